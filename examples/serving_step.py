"""A decoder served from a paged cache, with this library's operators end to end.

The model is small and random: two layers of 8 query heads on 2 key heads, block-scaled fp8 projections, a Q4_K
output matrix. What it does is what a server does in every step:

    quantize_fp8_b128, qmm_fp8_b128   the projections of the step's tokens
    kv_append                         their keys and values into their pages
    attn_paged                        prompts and single tokens of all sequences in one call
    qgemv_q4_k, token_logprobs        logits, the probability of the tokens that came, the alternatives
    kv_fork, kv_free, kv_compact      continuations of a sequence, its end, and a packed cache

`main` scores two prompts at once, the same tokens one by one, then three continuations of the first prompt before
and after the cache is packed, and prints how far the log probabilities are from those of a fresh start."""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_quantized_gemv_dequant_gb300 as qg  # noqa: E402
from bit_quantized_gemv_dequant_gb300 import synth  # noqa: E402

LAYERS, HIDDEN, HEADS, KV_HEADS, DIM, VOCAB, PAGE = 2, 512, 8, 2, 64, 1024, 16


def fp8_weight(w):
    """(codes, scales) of a weight [N, K], one scale per 128 x 128 values."""
    n, k = w.shape
    blocks = w.view(n // 128, 128, k // 128, 128)
    scales = blocks.abs().amax((1, 3)) / 448.0
    codes = (blocks / scales[:, None, :, None]).view(n, k).to(torch.float8_e4m3fn)
    return codes, scales.contiguous()


class Model:
    def __init__(self, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.embed = normal(VOCAB, HIDDEN)
        width = (HEADS + 2 * KV_HEADS) * DIM
        self.qkv = [fp8_weight(normal(width, HIDDEN) * HIDDEN**-0.5) for _ in range(LAYERS)]
        self.out = [fp8_weight(normal(HIDDEN, HEADS * DIM) * HIDDEN**-0.5) for _ in range(LAYERS)]
        self.head = torch.from_numpy(synth.q4_k_case(seed + 1, VOCAB, HIDDEN, 1)["w"]).cuda()


def linear(x, weight):
    codes, scales = qg.quantize_fp8_b128(x)
    return qg.qmm_fp8_b128(codes, scales, *weight)


def norm(x):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)


class Cache:
    """Pages of all layers' keys and values, and the sequences' rows in the page table."""

    def __init__(self, pages, width):
        self.planes = torch.zeros(LAYERS * 2, pages, KV_HEADS, PAGE, DIM, dtype=torch.bfloat16, device="cuda")
        self.table = torch.empty((0, width), dtype=torch.int32, device="cuda")
        self.lens = torch.empty(0, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")

    def add(self):
        row = torch.full((1, self.table.shape[1]), -1, dtype=torch.int32, device="cuda")
        self.table, self.lens = torch.cat([self.table, row]), torch.cat([self.lens, self.lens.new_zeros(1)])
        return self.table.shape[0] - 1

    def grow(self, counts):
        """Pages for counts[r] more tokens of each row, the lowest free ones; slots of the new tokens, row by row."""
        table, lens, refs = self.table.cpu(), self.lens.cpu(), self.refs.cpu()
        free, slots = iter((refs == 0).nonzero().flatten().tolist()), []
        for r, n in enumerate(counts):
            for t in range(int(lens[r]), int(lens[r]) + n):
                if table[r, t // PAGE] < 0:
                    page = next(free)
                    table[r, t // PAGE], refs[page] = page, 1
                slots.append(int(table[r, t // PAGE]) * PAGE + t % PAGE)
            lens[r] += n
        self.table, self.lens, self.refs = table.cuda(), lens.cuda(), refs.cuda()
        return torch.tensor(slots, dtype=torch.int64, device="cuda")

    def fork(self, parents):
        parents = torch.tensor(parents, dtype=torch.int32, device="cuda")
        table, lens, self.refs = qg.kv_fork(self.planes, self.table, self.lens, self.refs, parents, PAGE)
        first = self.table.shape[0]
        self.table, self.lens = torch.cat([self.table, table]), torch.cat([self.lens, lens])
        return list(range(first, self.table.shape[0]))

    def free(self, rows):
        drop = torch.zeros(self.table.shape[0], dtype=torch.uint8, device="cuda")
        drop[rows] = 1
        self.table, self.lens, self.refs = qg.kv_free(self.table, self.lens, self.refs, drop)

    def compact(self):
        self.table, self.refs, _, live = qg.kv_compact(self.planes, self.table, self.refs)
        return live


def step(model, cache, new):
    """Logits after each of the new tokens: new[r] lists those of row r (none is fine)."""
    counts = [len(t) for t in new]
    slots = cache.grow(counts)
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    x = model.embed[torch.tensor([t for row in new for t in row], device="cuda")]
    for layer in range(LAYERS):
        qkv = linear(norm(x), model.qkv[layer]).view(len(x), HEADS + 2 * KV_HEADS, DIM)
        k_cache, v_cache = cache.planes[2 * layer], cache.planes[2 * layer + 1]
        qg.kv_append(qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:], k_cache, v_cache, slots)
        heads = qg.attn_paged(qkv[:, :HEADS].to(torch.bfloat16), k_cache, v_cache, cache.table, offsets, cache.lens,
                              max_new=max(counts))
        x = x + linear(heads.view(len(x), HEADS * DIM), model.out[layer])
    return qg.qgemv_q4_k(model.head, norm(x).contiguous(), N=VOCAB)


def next_logprobs(logits, tokens):
    """Log probabilities of the tokens that follow, given the logits before each of them."""
    return qg.token_logprobs(logits, torch.tensor(tokens, device="cuda"), 5)


def score(model, tokens):
    """Log probabilities of tokens[1:] from a fresh cache, in one prefill."""
    cache = Cache(64, 16)
    cache.add()
    return next_logprobs(step(model, cache, [tokens])[:-1], tokens[1:])[0]


def main():
    model = Model()
    g = torch.Generator().manual_seed(7)
    a, b = (torch.randint(0, VOCAB, (n,), generator=g).tolist() for n in (75, 6))
    far = {}

    # two prompts of different lengths in one call, and each of them alone
    cache = Cache(64, 16)
    cache.add(), cache.add()
    logits = step(model, cache, [a, b])
    together = next_logprobs(torch.cat([logits[:74], logits[75:80]]), a[1:] + b[1:])[0]
    far["prompts together"] = (together - torch.cat([score(model, a), score(model, b)])).abs().max().item()

    # the shorter one, token by token
    single = Cache(64, 16)
    single.add()
    one = torch.cat([next_logprobs(step(model, single, [[t]]), [n])[0] for t, n in zip(b, b[1:])])
    far["token by token"] = (one - score(model, b)).abs().max().item()

    # three continuations of the first prompt, by its most likely next tokens
    best = next_logprobs(logits[74:75], [0])[4][0, :3].tolist()
    children = cache.fork([0, 0, 0])
    follow = torch.randint(0, VOCAB, (3,), generator=g).tolist()
    after = step(model, cache, [[], []] + [[t] for t in best])
    got = next_logprobs(after, follow)[0]
    want = torch.stack([score(model, a + [t, f])[-1] for t, f in zip(best, follow)])
    far["continuations"] = (got - want).abs().max().item()

    # one of them and the second prompt end; the cache is packed; the others go on
    cache.free([1, children[1]])
    live = int(cache.compact())
    assert live == cache.table[cache.table >= 0].unique().numel()
    again = step(model, cache, [[], [], [follow[0]], [], [follow[2]]])
    end = torch.randint(0, VOCAB, (2,), generator=g).tolist()
    got = next_logprobs(again, end)[0]
    want = torch.stack([score(model, a + [best[i], follow[i], e])[-1] for i, e in zip((0, 2), end)])
    far["after packing"] = (got - want).abs().max().item()
    assert qg.device_error() == 0
    return far


if __name__ == "__main__":
    for what, value in main().items():
        print("%-18s log probabilities differ by at most %.4f" % (what, value))
