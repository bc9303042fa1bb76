"""The serving operators, measured: the block-scaled 8-bit floating point product, attention of new tokens over
a paged cache, the upkeep of that cache's pages, and the log probabilities of given tokens.

A case is a dict of plain values. `prepare` makes what a user's program holds before the call, `run` makes the
call (the library's where `own` is true, elementary torch operations in 32 bits otherwise), `exact` computes the
same outputs from the definitions in 64 bits and `work` counts the bytes and operations that cannot be saved."""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token through a projection of the decode layer: latency and the weight's bytes
        dict(name="fp8 decode M=1", op="fp8", M=1, N=4096, K=4096, x="bf16", y="bf16"),
        # a small batch on a sharded layer: no size a multiple of a block, f32 on both sides
        dict(name="fp8 ragged M=37", op="fp8", M=37, N=2200, K=5200, x="f32", y="f32"),
        # a prompt through the widest projection of the decode layer: bound by the tensor cores
        dict(name="fp8 prefill M=4096", op="fp8", M=4096, N=12288, K=4096, x="bf16", y="bf16"),
        # one conversation, one token: the smallest call, all latency
        dict(name="attn one token", op="attn", B=1, new=1, new_low=1, ctx=700, ctx_low=700, Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16", softcap=0.0, window=0),
        # a serving batch of single tokens over contexts of very different lengths: bound by the cache's bytes
        dict(name="attn decode batch", op="attn", B=128, new=1, new_low=1, ctx=8192, ctx_low=65, Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16", softcap=0.0, window=0),
        # a mixed batch (idle slots, single tokens, short chunks) of a model with capped scores and a window
        dict(name="attn mixed capped window", op="attn", B=13, new=130, new_low=0, ctx=3001, ctx_low=40, Hq=20, Hkv=4,
             D=64, page=16, dtype="f16", softcap=30.0, window=1000),
        # two prompts in the middle of their prefill: 2048 new tokens each over a long cache
        dict(name="attn long chunks", op="attn", B=2, new=2048, new_low=2048, ctx=16384, ctx_low=8200, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16", softcap=0.0, window=0),
        # the keys and values of a step's tokens, parts of one fused f32 projection, into their pages
        dict(name="pages append", op="append", T=3001, Hq=32, Hkv=8, D=128, page=64, x="f32", dtype="bf16", skip=0.02),
        # a beam or sampling step: 16 conversations, three more continuations of each, over all layers' planes
        dict(name="pages fork", op="fork", B=16, copies=3, planes=32, pages=1500, P=128, len=4000, Hkv=8, D=128, page=32,
             dtype="bf16"),
        # conversations end and the cache is packed: a third of its pages free, all layers' planes
        dict(name="pages free and compact", op="compact", B=96, planes=24, pages=3000, P=64, len=1200, Hkv=8, D=128,
             page=32, dtype="bf16", freed=0.35),
        # the sampled token of one conversation, an odd vocabulary, part of it masked away
        dict(name="logprobs one token", op="logprobs", M=1, V=50021, pad=0, x="f32", top=20, masked=0.3, none=0),
        # scoring a prompt against a large vocabulary
        dict(name="logprobs prompt", op="logprobs", M=2048, V=131072, pad=0, x="bf16", top=5, masked=0.0, none=3),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["fp8", "fp8", "attn", "attn", "attn", "append", "fork", "compact", "logprobs", "logprobs"])
    if op == "fp8":
        M, N = log(1, 4096), log(64, 12288)
        x = rng.choice(["bf16", "f32", "f16"])
        return dict(op=op, M=M, N=N, K=16 * log(4, 256) if rng.random() < 0.8 else log(33, 2000), x=x,
                    y=rng.choice(["bf16", "f32"]))
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8])
        kind = rng.choice(["decode", "mixed", "chunk"])
        if kind == "decode":
            B, new, low, ctx = log(1, 128), 1, 1, log(1, 8192)
        elif kind == "mixed":
            B, new, low, ctx = log(2, 24), log(2, 300), 0, log(300, 4000)
        else:
            B, new = log(1, 3), log(64, 1500)
            low, ctx = new, log(max(new, 200), 10000)
        ctx = max(ctx, new)
        return dict(op=op, B=B, new=new, new_low=low, ctx=ctx, ctx_low=log(1, ctx), Hq=Hkv * rng.choice([r for r in (1, 2, 4, 5, 8) if r * Hkv <= 32]),
                    Hkv=Hkv, D=rng.choice([64, 128, 128]), page=rng.choice([8, 16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "f16"]), softcap=rng.choice([0.0, 0.0, 30.0]),
                    window=rng.choice([0, 0, log(1, 2000)]))
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, T=log(1, 3001), Hq=rng.choice([0, 4 * Hkv]), Hkv=Hkv, D=rng.choice([64, 128]),
                    page=rng.choice([8, 16, 32, 64, 128]), x=rng.choice(["f32", "bf16", "f16"]),
                    dtype=rng.choice(["bf16", "f16"]), skip=rng.choice([0.0, 0.1]))
    if op == "fork":
        B, length, page = log(1, 16), log(1, 3000), rng.choice([8, 16, 32])
        P = -(-length // page) + rng.randint(0, 9)
        return dict(op=op, B=B, copies=rng.randint(1, 3), planes=log(1, 32), pages=B * (P + 3) + rng.randint(0, 200), P=P,
                    len=length, Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=page,
                    dtype=rng.choice(["bf16", "f16"]))
    if op == "compact":
        B, length, page = log(1, 96), log(1, 1000), rng.choice([8, 16, 32])
        P = -(-length // page) + rng.randint(0, 9)
        return dict(op=op, B=B, planes=log(1, 24), pages=int(B * -(-length // page) * rng.uniform(1.0, 1.3)) + 1, P=P,
                    len=length, Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=page,
                    dtype=rng.choice(["bf16", "f16"]), freed=round(rng.uniform(0.1, 0.9), 2))
    V = log(40, 131072)
    M = max(1, min(2048, log(1, 4096)))
    return dict(op=op, M=M, V=V, pad=rng.choice([0, 0, rng.randint(1, 64)]), x=rng.choice(["f32", "bf16", "f16"]),
                top=rng.choice([0, 1, 5, 20, 32]), masked=rng.choice([0.0, 0.5]), none=rng.choice([0, 0, 1]))


def spread(low, high, n, turn=0):
    """n whole numbers from low to high, evenly spaced, in an order that mixes small and large ones."""
    if n == 1:
        return [high]
    v = [low + (high - low) * i // (n - 1) for i in range(n)]
    step = next(s for s in range(max(1, n * 5 // 8), 2 * n + 2) if math.gcd(s, n) == 1)
    return [v[(i * step + turn) % n] for i in range(n)]


def lengths(c):
    """The new tokens and the context (the new ones included) of each sequence of an attention case."""
    new = spread(c["new_low"], c["new"], c["B"])
    ctx = [max(n, t) for n, t in zip(new, spread(c["ctx_low"], c["ctx"], c["B"], 1))]
    return new, ctx


# ------------------------------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    return globals()["prepare_" + case["op"]](case, torch.Generator("cuda").manual_seed(seed))


def normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def prepare_fp8(c, g):
    M, N, K = c["M"], c["N"], c["K"]
    # activations: unit variance with a few channels that stand out, as after a norm
    x = normal(g, M, K) * torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 12.0, 1.0)
    nb, kb = -(-N // 128), -(-K // 128)
    w = torch.zeros(nb * 128, kb * 128, device="cuda")
    w[:N, :K] = normal(g, N, K) * 0.02
    blocks = w.view(nb, 128, kb, 128)
    w_scales = blocks.abs().amax((1, 3)) / 448.0
    codes = (blocks / w_scales[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * 128, kb * 128)
    return dict(c, x=x.to(DTYPES[c["x"]]), w=codes.view(torch.uint8)[:N, :K].contiguous().view(torch.float8_e4m3fn),
                w_scales=w_scales.contiguous())


def prepare_attn(c, g):
    new, ctx = lengths(c)
    B, page, dt = c["B"], c["page"], DTYPES[c["dtype"]]
    counts = [-(-t // page) for t in ctx]
    total = sum(counts)
    num_pages, P = total + total // 8 + 1, max(counts) + 1
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    table, at = np.full((B, P), -1, np.int32), 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    k = normal(g, num_pages, c["Hkv"], page, c["D"], dtype=dt)
    v = normal(g, num_pages, c["Hkv"], page, c["D"], dtype=dt)
    # pages that are not in use, and the end of each sequence's last page, hold what memory happens to hold
    for t in (k, v):
        t[torch.from_numpy(order[total:].astype(np.int64)).cuda()] = float("nan")
    ends = [(int(table[b, n - 1]), ctx[b] - (n - 1) * page) for b, n in enumerate(counts) if n]
    last = torch.tensor([p for p, _ in ends], device="cuda")
    used = torch.tensor([u for _, u in ends], device="cuda")
    dead = torch.arange(page, device="cuda")[None, :] >= used[:, None]
    for t in (k, v):
        t[last] = torch.where(dead[:, None, :, None], torch.full((), float("nan"), dtype=dt, device="cuda"), t[last])
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    return dict(c, q=normal(g, sum(new), c["Hq"], c["D"], dtype=dt), k=k, v=v, table=torch.from_numpy(table).cuda(),
                offsets=offsets, lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"))


def prepare_append(c, g):
    T, page = c["T"], c["page"]
    num_pages = -(-T // page) * 2 + 1
    dt = DTYPES[c["dtype"]]
    qkv = normal(g, T, c["Hq"] + 2 * c["Hkv"], c["D"], dtype=DTYPES[c["x"]])
    slots = torch.randperm(num_pages * page, generator=g, device="cuda")[:T].clone()
    slots[torch.rand(T, generator=g, device="cuda") < c["skip"]] = -1  # padding tokens
    k_cache = normal(g, num_pages, c["Hkv"], page, c["D"], dtype=dt)
    v_cache = normal(g, num_pages, c["Hkv"], page, c["D"], dtype=dt)
    return dict(c, k=qkv[:, c["Hq"]:c["Hq"] + c["Hkv"]], v=qkv[:, c["Hq"] + c["Hkv"]:], slots=slots, k_cache=k_cache,
                v_cache=v_cache)


def prepare_pages(c, g, shared):
    """A cache with B conversations in it, their pages spread all over; the first `shared` of them share a page."""
    page, lens = c["page"], spread(max(1, c["len"] // 3), c["len"], c["B"])
    order = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32).cpu().numpy()
    table, refs, at = np.full((c["B"], c["P"]), -1, np.int32), np.zeros(c["pages"], np.int32), 0
    for b, n in enumerate(-(-t // page) for t in lens):
        table[b, :n] = order[at:at + n]
        at += n
        if 0 < b < shared:
            table[b, 0] = table[0, 0]  # a common prompt: its first page is held once
        np.add.at(refs, table[b, :n], 1)
    cache = normal(g, c["planes"], c["pages"], c["Hkv"], page, c["D"], dtype=DTYPES[c["dtype"]])
    return dict(c, cache=cache, table=torch.from_numpy(table).cuda(), refs=torch.from_numpy(refs).cuda(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def prepare_fork(c, g):
    parents = torch.arange(c["B"], device="cuda", dtype=torch.int32).repeat(c["copies"])
    return dict(prepare_pages(c, g, 1), parents=parents[torch.randperm(parents.numel(), generator=g, device="cuda")])


def prepare_compact(c, g):
    gone = torch.zeros(c["B"], dtype=torch.uint8, device="cuda")
    gone[torch.randperm(c["B"], generator=g, device="cuda")[:round(c["B"] * c["freed"])]] = 1
    return dict(prepare_pages(c, g, 3), gone=gone)


def prepare_logprobs(c, g):
    M, V = c["M"], c["V"]
    x = normal(g, M, V + c["pad"]) * 3.0
    if c["masked"]:
        x.masked_fill_(torch.rand(M, V + c["pad"], generator=g, device="cuda") < c["masked"], float("-inf"))
    targets = torch.randint(0, V, (M,), generator=g, device="cuda")
    if c["none"] and M > 2:
        x[1] = float("-inf")  # a mask that leaves nothing
        targets[torch.randperm(M, generator=g, device="cuda")[:c["none"]]] = -1  # positions without a token
    return dict(c, x=x.to(DTYPES[c["x"]])[:, :V], targets=targets)


# --------------------------------------------------------------------------------------------------- the calls
def run(state):
    return globals()[("own_" if own else "plain_") + state["op"]](state)


def own_fp8(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    codes, scales = qg.quantize_fp8_b128(s["x"])
    return {"y": qg.qmm_fp8_b128(codes, scales, s["w"], s["w_scales"], out_dtype=DTYPES[s["y"]]), "scales": scales}


def plain_fp8(s):
    x = s["x"].float()
    M, K = x.shape
    N, kb = s["w"].shape[0], -(-K // 128)
    pad = kb * 128 - K
    x = torch.cat([x, x.new_zeros(M, pad)], 1).view(M, kb, 128)
    scales = x.abs().amax(2) / torch.full((), 448.0, device=x.device)
    scales = torch.where(scales > 0, scales, torch.ones_like(scales))
    a = ((x / scales[:, :, None]).to(torch.float8_e4m3fn).float() * scales[:, :, None]).view(M, kb * 128)[:, :K]
    w = s["w"].float() * s["w_scales"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return {"y": (a @ w.t()).to(DTYPES[s["y"]]), "scales": scales}


def own_attn(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    out, lse = qg.attn_paged(s["q"], s["k"], s["v"], s["table"], s["offsets"], s["lens"], max_new=s["new"],
                             softcap=s["softcap"], window=s["window"], return_lse=True)
    return {"out": out, "lse": lse}


def plain_attn(s):
    T, Hq, D = s["q"].shape
    B, Hkv, new, group = s["B"], s["Hkv"], s["new"], Hq // s["Hkv"]
    dev = s["q"].device
    at, lens = s["offsets"].long(), s["lens"].long()
    count = at[1:] - at[:-1]
    table = s["table"].clamp(min=0).long()
    L = table.shape[1] * s["page"]
    held = torch.arange(L, device=dev)[None, :] < lens[:, None]  # [B, L]
    k = s["k"][table].float().transpose(1, 2).reshape(B, Hkv, L, D)
    v = s["v"][table].float().transpose(1, 2).reshape(B, Hkv, L, D)
    v = torch.where(held[:, None, :, None], v, 0.0)
    j = torch.arange(new, device=dev)
    real = j[None, :] < count[:, None]  # [B, new]
    row = (at[:-1, None] + j[None, :]).clamp(max=T - 1)
    q = s["q"].float()[row].view(B, new, Hkv, group, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, group * new, D)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, group, new, L) * (1.0 / math.sqrt(D))
    if s["softcap"] > 0:
        x = torch.tanh(x / s["softcap"]) * s["softcap"]
    pos = (lens - count)[:, None] + j[None, :]
    seen = torch.arange(L, device=dev)[None, None, :] <= pos[:, :, None]
    if s["window"]:
        seen &= torch.arange(L, device=dev)[None, None, :] > pos[:, :, None] - s["window"]
    x = torch.where((seen & held[:, None, :])[:, None, None], x, float("-inf"))
    top = x.amax(4, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - top)
    total = p.sum(4, keepdim=True)
    o = torch.matmul((p / total).view(B, Hkv, group * new, L), v).view(B, Hkv, group, new, D)
    lse = (top + torch.log(total)).squeeze(4)
    out = o.permute(0, 3, 1, 2, 4).reshape(B, new, Hq, D)[real]
    return {"out": out.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(B, new, Hq)[real]}


def own_append(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    qg.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
    return {"k": s["k_cache"], "v": s["v_cache"]}


def plain_append(s):
    live = s["slots"] >= 0
    at = s["slots"][live]
    page, place = at // s["page"], at % s["page"]
    s["k_cache"][page, :, place] = s["k"][live].to(s["k_cache"].dtype)
    s["v_cache"][page, :, place] = s["v"][live].to(s["v_cache"].dtype)
    return {"k": s["k_cache"], "v": s["v_cache"]}


def own_fork(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    table, lens, refs = qg.kv_fork(s["cache"], s["table"], s["lens"], s["refs"], s["parents"], s["page"])
    return {"table": table, "lens": lens, "refs": refs, "cache": s["cache"]}


def plain_fork(s):
    parents = s["parents"].long()
    lens = s["lens"][parents]
    whole, part = (lens // s["page"]).long(), lens % s["page"] > 0
    col = torch.arange(s["P"], device=lens.device)[None, :]
    old = s["table"][parents]
    free = (s["refs"] == 0).nonzero().squeeze(1)[:parents.numel()].to(torch.int32)
    fresh = free[(part.cumsum(0) - 1).clamp(min=0)]
    table = torch.where(col < whole[:, None], old, -1)
    table = torch.where((col == whole[:, None]) & part[:, None], fresh[:, None], table)
    refs = s["refs"] + torch.bincount(table[table >= 0], minlength=s["pages"]).to(torch.int32)
    src = old.gather(1, whole[:, None].clamp(max=s["P"] - 1)).squeeze(1)[part].long()
    s["cache"][:, fresh[part].long()] = s["cache"][:, src]
    return {"table": table, "lens": lens, "refs": refs, "cache": s["cache"]}


def own_compact(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    table, lens, refs = qg.kv_free(s["table"], s["lens"], s["refs"], s["gone"])
    table, refs, moved, live = qg.kv_compact(s["cache"], table, refs)
    return {"table": table, "lens": lens, "refs": refs, "moved": moved, "live": live, "cache": s["cache"]}


def plain_compact(s):
    gone = s["gone"] > 0
    dropped = s["table"][gone]
    refs = s["refs"] - torch.bincount(dropped[dropped >= 0], minlength=s["pages"]).to(torch.int32)
    table = torch.where(gone[:, None], -1, s["table"])
    lens = torch.where(gone, 0, s["lens"])
    held = refs > 0
    live = held.sum()
    page = torch.arange(s["pages"], device=refs.device)
    src, dst = page[held & (page >= live)], page[~held & (page < live)]
    moved = torch.where(held, page, -1).to(torch.int32)
    moved[src] = dst.to(torch.int32)
    s["cache"][:, dst] = s["cache"][:, src]
    packed = torch.zeros_like(refs)
    packed[moved[held].long()] = refs[held]
    table = torch.where(table >= 0, moved[table.clamp(min=0).long()], -1)
    return {"table": table, "lens": lens, "refs": packed, "moved": moved, "live": live.to(torch.int32).view(1),
            "cache": s["cache"]}


def own_logprobs(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    picked, entropy, rank, top, ids = qg.token_logprobs(s["x"], s["targets"], s["top"])
    return {"picked": picked, "entropy": entropy, "rank": rank, "top": top, "ids": ids}


def plain_logprobs(s):
    x = s["x"].float()
    M, V = x.shape
    m = x.amax(1, keepdim=True).clamp(min=-3.4e38)
    e = torch.exp(x - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)  # -inf where the mask left nothing
    logp = torch.where(torch.isinf(x), x, (x - m) - torch.log(total))
    entropy = -torch.where(e > 0, e / total * logp, 0.0).sum(1)
    given = s["targets"] >= 0
    t = s["targets"].clamp(min=0)[:, None]
    rank = torch.where(given, (x > x.gather(1, t)).sum(1), -1).to(torch.int32)
    picked = torch.where(given, logp.gather(1, t).squeeze(1), 0.0)
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(2**31) - bits - 1, bits) * 2**32 + (2**32 - 1 - torch.arange(V, device=x.device))
    ids = (2**32 - 1 - torch.topk(key, min(s["top"], V), dim=1).values % 2**32)
    return {"picked": picked, "entropy": torch.where(torch.isinf(lse.squeeze(1)), 0.0, entropy), "rank": rank,
            "top": logp.gather(1, ids), "ids": ids.to(torch.int32)}


# --------------------------------------------------------------------------------------------- the definitions
def exact(case, seed):
    f = globals().get("exact_" + case["op"])
    return f(prepare(case, seed)) if f else None


def round_e4m3(v):
    """The nearest e4m3 value of each (ties to even), by arithmetic: 4 significant bits, steps of 2**-9 at least."""
    _, e = torch.frexp(v)
    step = torch.exp2(torch.clamp(e - 4, min=-9).double())
    return torch.round(v / step).mul(step).clamp(-448.0, 448.0)


def exact_fp8(s):
    x, w = s["x"].double(), s["w"].double()
    (M, K), N = x.shape, w.shape[0]
    y = torch.zeros(M, N, dtype=torch.float64, device=x.device)
    scales = torch.ones(M, -(-K // 128), dtype=torch.float64, device=x.device)
    for b in range(-(-K // 128)):
        part = x[:, b * 128:(b + 1) * 128]
        top = part.abs().amax(1)
        # scale and quotient are f32 numbers by definition: the code is the e4m3 value nearest to the rounded quotient
        scale = torch.where(top > 0, (top / 448.0).float().double(), 1.0)
        scales[:, b] = scale
        per_row = s["w_scales"][:, b].double()[torch.arange(N, device=x.device) // 128]
        product = round_e4m3((part / scale[:, None]).float().double()) @ w[:, b * 128:(b + 1) * 128].t()
        y += product * scale[:, None] * per_row[None, :]
    return {"y": y, "scales": scales}


def exact_attn(s):
    at, outs, sums = s["offsets"].tolist(), [], []
    group, D = s["Hq"] // s["Hkv"], s["D"]
    for b, n in enumerate(s["lens"].tolist()):
        count = at[b + 1] - at[b]
        if not count:
            continue
        pages = s["table"][b, :-(-n // s["page"])].long()
        k = s["k"][pages].double().transpose(0, 1).reshape(s["Hkv"], -1, D)[:, :n]
        v = s["v"][pages].double().transpose(0, 1).reshape(s["Hkv"], -1, D)[:, :n]
        pos = torch.arange(n - count, n, device=k.device)[:, None]
        key = torch.arange(n, device=k.device)[None, :]
        hidden = (key > pos) | (key <= pos - s["window"]) if s["window"] else key > pos
        o = torch.empty(count, s["Hq"], D, dtype=torch.float64, device=k.device)
        l = torch.empty(count, s["Hq"], dtype=torch.float64, device=k.device)
        for h in range(s["Hq"]):
            x = s["q"][at[b]:at[b + 1], h].double() @ k[h // group].t() / math.sqrt(D)
            x = s["softcap"] * torch.tanh(x / s["softcap"]) if s["softcap"] > 0 else x
            x = x.masked_fill_(hidden, -math.inf)
            l[:, h] = torch.logsumexp(x, 1)
            o[:, h] = torch.softmax(x, 1) @ v[h // group]
        outs.append(o)
        sums.append(l)
    if not outs:
        return {"out": s["q"].double(), "lse": s["q"].double()[..., 0]}
    return {"out": torch.cat(outs), "lse": torch.cat(sums)}


def exact_logprobs(s):
    picked, entropy, top = [], [], []
    for x, t in zip(s["x"].split(64), s["targets"].split(64)):
        x = x.double()
        empty = torch.isinf(x).all(1)
        logp = torch.where(empty[:, None], x, torch.log_softmax(x, 1))
        picked.append(torch.where(t >= 0, logp.gather(1, t.clamp(min=0)[:, None]).squeeze(1), 0.0))
        entropy.append(torch.where(empty, 0.0, torch.special.entr(torch.exp(logp)).sum(1)))
        top.append(torch.sort(logp, 1, descending=True).values[:, :s["top"]])
    return {"picked": torch.cat(picked), "entropy": torch.cat(entropy), "rank": None, "top": torch.cat(top), "ids": None}


# -------------------------------------------------------------------------------------------------- the floors
def work(case):
    return globals()["work_" + case["op"]](case)


def work_fp8(c):
    M, N, K = c["M"], c["N"], c["K"]
    nb, kb = -(-N // 128), -(-K // 128)
    return {"bytes": M * K * SIZE[c["x"]] + N * K + 4 * (nb + M) * kb + M * N * SIZE[c["y"]], "flops": 2 * M * N * K}


def work_attn(c):
    new, ctx = lengths(c)
    keys = reads = 0
    for n, t in zip(new, ctx):
        w = c["window"] or t
        pos = np.arange(t - n, t)
        keys += int(np.minimum(pos + 1, w).sum())
        reads += min(t, n - 1 + w) if n else 0
    one = c["D"] * SIZE[c["dtype"]]
    return {"bytes": 2 * reads * c["Hkv"] * one + 2 * sum(new) * c["Hq"] * one + 4 * sum(new) * c["Hq"],
            "flops": 4 * keys * c["Hq"] * c["D"]}


def work_append(c):
    n = c["T"] * c["Hkv"] * c["D"] * 2
    return {"bytes": n * (SIZE[c["x"]] + SIZE[c["dtype"]]) + 8 * c["T"], "flops": 0}


def page_bytes(c):
    return c["planes"] * c["Hkv"] * c["page"] * c["D"] * SIZE[c["dtype"]]


def work_fork(c):
    lens = spread(max(1, c["len"] // 3), c["len"], c["B"])
    fresh = c["copies"] * sum(1 for t in lens if t % c["page"])
    return {"bytes": 2 * fresh * page_bytes(c) + 8 * c["pages"] + 8 * c["B"] * c["copies"] * c["P"], "flops": 0}


def work_compact(c):
    counts = [-(-t // c["page"]) for t in spread(max(1, c["len"] // 3), c["len"], c["B"])]
    live = sum(counts) * (1.0 - round(c["B"] * c["freed"]) / c["B"])
    # of evenly spread live pages those past the number of live ones move
    moves = live * max(0.0, 1.0 - live / c["pages"])
    return {"bytes": int(2 * moves * page_bytes(c)) + 12 * c["pages"] + 16 * c["B"] * c["P"], "flops": 0}


def work_logprobs(c):
    return {"bytes": c["M"] * c["V"] * SIZE[c["x"]] + c["M"] * (8 + 12 + 8 * min(c["top"], c["V"])), "flops": 4 * c["M"] * c["V"]}
