"""The serving operators' calls as a program makes them: under transforms, from several threads, in several graphs and
among calls that overlap."""
import concurrent.futures
import os
import subprocess
import sys

import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg
from bit_quantized_gemv_dequant_gb300 import synth

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_tensor_without_data_raises():
    """Tensors inside torch.vmap have no address: an error, after which the process goes on."""
    code = """
import torch
import bit_quantized_gemv_dequant_gb300 as qg
x = torch.ones(3, 4, 256, device="cuda")
for i in range(2):
    try:
        torch.vmap(lambda x: qg.quantize_fp8_b128(x))(x)
    except RuntimeError:
        print("raised")
codes, scales = qg.quantize_fp8_b128(x[0])
assert (codes.float() == 448).all() and qg.device_error() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["raised", "raised"], (r.returncode, r.stdout, r.stderr[-2000:])


def attention(seed, lens=(900, 70, 1300), new=(1, 1, 1)):
    """A call's arguments: sequences that several CTAs share, so that parts meet in the scratch."""
    g = torch.Generator("cuda").manual_seed(seed)
    counts = [-(-n // 16) for n in lens]
    pages = sum(counts)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(counts)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    k, v = (torch.randn(pages, 2, 16, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(sum(new), 8, 64, generator=g, device="cuda").bfloat16()
    offsets = torch.tensor([0] + list(new), device="cuda").cumsum(0).to(torch.int32)
    return q, k, v, table, offsets, torch.tensor(lens, dtype=torch.int32, device="cuda")


def in_threads(work, n):
    """[work(0), ... work(n - 1)], each by a thread of its own; an exception in one is raised here."""
    with concurrent.futures.ThreadPoolExecutor(n) as pool:
        return [f.result() for f in [pool.submit(work, i) for i in range(n)]]


class Fork:
    """A cache of four planes with five rows of 40 tokens, and a fork of them."""

    def __init__(self, seed, children):
        g = torch.Generator("cuda").manual_seed(seed)
        self.cache = torch.randint(-999, 999, (4, 64, 16, 8), generator=g, device="cuda", dtype=torch.int32)
        order = torch.randperm(64, generator=g, device="cuda").to(torch.int32)
        self.table = order[:15].view(5, 3).contiguous()
        self.refs = torch.zeros(64, dtype=torch.int32, device="cuda")
        self.refs[self.table.flatten().long()] = 1
        self.lens = torch.full((5,), 40, dtype=torch.int32, device="cuda")
        self.parents = torch.randint(0, 5, (children,), generator=g, device="cuda").to(torch.int32)

    def __call__(self):
        return qg.kv_fork(self.cache, self.table, self.lens, self.refs, self.parents, 16)

    def right(self, out):
        """Each child's last page is a copy of its parent's."""
        table, lens, _ = out
        fresh, old = table[:, 2].long(), self.table[self.parents.long(), 2].long()
        return bool((lens == 40).all()) and torch.equal(self.cache[:, fresh], self.cache[:, old])


def test_two_threads_on_one_stream():
    """Each call's two kernels pass data through the stream's scratch: no other thread's come between them."""
    args = [attention(1), attention(2, (40, 1500, 300), (30, 1, 50))]
    want = [qg.attn_paged(*a) for a in args]
    forks = [Fork(3, 7), Fork(4, 11)]

    def work(i):
        torch.cuda.synchronize()
        wrong = 0
        for _ in range(200):
            wrong += not torch.equal(qg.attn_paged(*args[i]), want[i])
            forks[i].cache[:, :, :] = forks[i].cache.flip(0)  # other contents every time
            wrong += not forks[i].right(forks[i]())
        return wrong

    assert in_threads(work, 2) == [0, 0] and qg.device_error() == 0


def test_first_call_of_a_thread():
    """A thread that has done nothing on the device before."""
    one, chunk = attention(5), attention(6, (400, 90), (200, 20))
    codes = [torch.randn(m, 512, device="cuda").to(torch.float8_e4m3fn) for m in (3, 700, 300)]
    scales = [torch.ones(m, 4, device="cuda") for m in (3, 700, 3)]
    calls = [lambda: qg.attn_paged(*one, max_new=1), lambda: qg.attn_paged(*chunk)]
    calls += [lambda i=i: qg.qmm_fp8_b128(codes[i], scales[i], codes[2], scales[2]) for i in range(2)]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        assert torch.equal(in_threads(lambda i: call(), 1)[0], want)


def captured(call):
    """A graph of 20 calls, captured on the stream that torch.cuda.graph takes by default, and the last one's result."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            out = call()
    return graph, out


def test_graphs_beside_each_other():
    """Two graphs replayed at the same time on two streams, with eager calls on a third."""
    args = [attention(7), attention(8, (40, 1500, 300), (30, 1, 50)), attention(9, (800, 600), (1, 1))]
    want = [qg.attn_paged(*a) for a in args]
    forks = [Fork(10, 7), Fork(11, 11)]
    made = [captured(lambda a=a: qg.attn_paged(*a)) for a in args[:2]]
    made_forks = [captured(f) for f in forks]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(30):
        for (_, out), f in zip(made, forks):
            out.zero_()
            f.cache.copy_(f.cache.flip(0))
        torch.cuda.synchronize()
        for s, (graph, _), (fork, _) in zip(streams, made, made_forks):
            with torch.cuda.stream(s):
                graph.replay()
                fork.replay()
        eager = [qg.attn_paged(*args[2]) for _ in range(10)]
        torch.cuda.synchronize()
        assert all(torch.equal(out, w) for (_, out), w in zip(made, want))
        assert all(torch.equal(out, want[2]) for out in eager)
        assert all(f.right(out) for f, (_, out) in zip(forks, made_forks))
    assert qg.device_error() == 0


@pytest.fixture
def pdl():
    """Sets QG_OPT_PDL; it is what it was afterwards."""
    old = qg.get_option(qg.QG_OPT_PDL)
    yield lambda value: qg.set_option(qg.QG_OPT_PDL, value)
    qg.set_option(qg.QG_OPT_PDL, old)


def projection(seed, n, k):
    w = torch.from_numpy(synth.q4_k_case(seed, 64, k, 1)["w"]).cuda()
    return w.flatten().repeat(n // 64)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_serving_after_independent_projections(pdl, mode):
    """Projections that need not wait for each other, then a call that reads what all of them wrote."""
    n, parts = 16384, 3
    ws = [projection(20 + i, n, 4096) for i in range(parts)]
    g = torch.Generator("cuda").manual_seed(21)
    xs = [torch.randn(1, 4096, generator=g, device="cuda") for _ in range(12)]
    targets = torch.randint(0, n * parts, (1,), generator=g, device="cuda")
    logits = torch.empty(1, n * parts, device="cuda")
    pieces = [logits[:, i * n:(i + 1) * n] for i in range(parts)]

    def step(x, mode):
        pdl(mode)
        for w, piece in zip(ws, pieces):
            qg.qgemv_q4_k(w, x, piece, N=n)
        return qg.token_logprobs(logits, targets, 5)

    want = [step(x, 0) for x in xs]
    got = [step(x, mode) for x in xs]
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert qg.device_error() == 0


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_independent_projection_after_serving(pdl, mode):
    """A projection that has nothing to do with the serving call before it, but with what came before that."""
    n, k = 4096, 4096
    w = projection(30, n, k)
    g = torch.Generator("cuda").manual_seed(31)
    big = torch.randn(4096, 4096, generator=g, device="cuda")
    x = torch.empty(1, k, device="cuda")
    args = attention(32)
    fork, codes = Fork(33, 7), torch.ones(2, 512, device="cuda").to(torch.float8_e4m3fn)
    small = torch.randn(3, 5000, generator=g, device="cuda")
    rows, one = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.ones(2, 4, device="cuda")
    pair = torch.arange(2, dtype=torch.int32, device="cuda")
    serving = [lambda: qg.attn_paged(*args, max_new=1), lambda: qg.attn_paged(*args, max_new=40), fork,
               lambda: qg.kv_copy_pages(fork.cache, pair, pair + 2), lambda: qg.qmm_fp8_b128(codes, one, codes, one[:1]),
               lambda: qg.qmm_fp8_b128(codes.repeat(80, 1), one.repeat(80, 1), codes, one[:1]),
               lambda: qg.token_logprobs(small, rows, 3)]

    def run(mode):
        out = []
        for i, call in enumerate(serving):
            pdl(0)
            v = torch.full((4096, 1), 0.01 * (i + 1), device="cuda")
            for _ in range(3):
                v = torch.mm(big, v) / 64
            torch.mm(v.t(), big, out=x)  # (some time on the way, so that a call that does not wait reads the old x)
            call()
            pdl(mode)
            out.append(qg.qgemv_q4_k(w, x, N=n))
        return out

    want = run(0)
    for a, b in zip(want, run(mode)):
        assert torch.equal(a, b)
    assert qg.device_error() == 0


def chain():
    """Steps in which every call reads what the one before wrote, without a pause: the results of all of them."""
    q, k, v, table, offsets, lens = attention(40, (900, 70, 1300), (1, 30, 1))
    g = torch.Generator("cuda").manual_seed(41)
    w = torch.randn(512, 512, generator=g, device="cuda").to(torch.float8_e4m3fn)
    head = torch.randn(5000, 512, generator=g, device="cuda").to(torch.float8_e4m3fn)
    one, many = torch.ones(4, 4, device="cuda"), torch.ones(40, 4, device="cuda")
    targets = torch.randint(0, 5000, (32,), generator=g, device="cuda")
    last = torch.tensor([n - 1 for n, c in ((900, 1), (70, 30), (1300, 1)) for _ in range(c)], device="cuda")
    row = torch.tensor([0] + [1] * 30 + [2], device="cuda")
    slots = table.long()[row, last // 16] * 16 + last % 16
    slots[1:30] = -1
    out = []
    for _ in range(20):
        a, lse = qg.attn_paged(q, k, v, table, offsets, lens, max_new=30, return_lse=True)
        codes, scales = qg.quantize_fp8_b128(a.view(32, 512))
        x = qg.qmm_fp8_b128(codes, scales, w, one, out_dtype=torch.bfloat16)
        q = x.view(32, 8, 64)
        qg.kv_append(q[:, :2], q[:, 2:4], k, v, slots)
        codes, scales = qg.quantize_fp8_b128(x)
        out += [a, lse, x, *qg.token_logprobs(qg.qmm_fp8_b128(codes, scales, head, many), targets, 3)]
    torch.cuda.synchronize()
    return [t.cpu() for t in out]


def test_overlapped_calls_give_the_same(pdl, tmp_path):
    """In a process where QG_OPT_PDL has never been 2, calls start while the one before ends; here they do not."""
    code = "import sys, torch; sys.path[:0] = ['tests', '.']; import test_gpu_serving_calls as t; torch.save(t.chain(), sys.argv[1])"
    r = subprocess.run([sys.executable, "-c", code, str(tmp_path / "out.pt")], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    pdl(2)
    pdl(0)
    for a, b in zip(torch.load(tmp_path / "out.pt"), chain(), strict=True):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert qg.device_error() == 0


def test_arguments_that_are_no_streams_or_truth_values():
    x, args = torch.ones(2, 128, device="cuda"), attention(50)
    with pytest.raises(OverflowError):
        qg.quantize_fp8_b128(x, stream=1 << 200)
    with pytest.raises(AttributeError):
        qg.quantize_fp8_b128(x, stream="0")
    with pytest.raises(RuntimeError):  # a tensor of several values
        qg.attn_paged(*args, return_lse=x)
    assert qg.quantize_fp8_b128(x, stream=0)[1].shape == (2, 1)


def test_first_call_of_a_thread_is_captured():
    args = attention(60)
    want = qg.attn_paged(*args)
    torch.cuda.synchronize()

    def work(_):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = qg.attn_paged(*args)
        graph.replay()
        torch.cuda.synchronize()
        return out

    assert torch.equal(in_threads(work, 1)[0], want)
