"""The operators between a layer's products as a program calls them: one after the other through a layer, in graphs
that run beside each other, from several threads, on other streams and among calls that overlap. Every step of a layer is
held against its definition on the step's own inputs, with the bounds of the operators' tests."""
import subprocess
import sys

import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg
import test_gpu_rms_norm as norms
import test_gpu_rope as rope
import test_gpu_silu_mul as gates
from test_gpu_fp8 import E4M3, check_product, codes_like, rng, scales_like
from test_gpu_grouped import Case as Experts
from test_gpu_serving_calls import ROOT, captured, in_threads, pdl, projection  # noqa: F401

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV_HEADS, DIM, PAGE, WIDE, COUNT = 512, 8, 2, 64, 16, 384, 6


def weight(g, n, k, *lead):
    """(codes, scales) with products of unit inputs near 1."""
    codes = (torch.randn(*lead, n, k, generator=g, device="cuda") * 80).clamp(-448, 448).to(E4M3)
    scales = (torch.rand(*lead, -(-n // 128), -(-k // 128), generator=g, device="cuda") + 0.5) / (80 * k**0.5)
    return codes, scales


class Layer:
    """A decoder layer with experts, its cache, and the tokens of a step: sequences of 900 and 70 keys with 1 and 30 new
    ones, and one that has just begun."""

    def __init__(self, seed):
        g = rng(seed)
        self.lens, self.new = [900, 70, 5], [1, 30, 5]
        T = sum(self.new)
        self.x = torch.randn(T, HIDDEN, generator=g, device="cuda").bfloat16()
        self.residual = torch.randn(T, HIDDEN, generator=g, device="cuda")
        self.norms = [torch.rand(HIDDEN, generator=g, device="cuda").bfloat16() + 0.5 for _ in range(2)]
        self.qkv = weight(g, (HEADS + 2 * KV_HEADS) * DIM, HIDDEN)
        self.out = weight(g, HIDDEN, HEADS * DIM)
        self.up, self.down = weight(g, 2 * WIDE, HIDDEN, COUNT), weight(g, HIDDEN, WIDE, COUNT)
        counts = [-(-n // PAGE) for n in self.lens]
        order = torch.randperm(sum(counts) + 3, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((3, max(counts)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = [torch.randn(len(order), KV_HEADS, PAGE, DIM, generator=g, device="cuda").bfloat16() for _ in range(2)]
        self.offsets = torch.tensor([0] + self.new, device="cuda").cumsum(0).to(torch.int32)
        self.context = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.positions = torch.cat([torch.arange(n - c, n, device="cuda") for n, c in zip(self.lens, self.new)])
        row = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(self.new, device="cuda"))
        self.slots = self.table.long()[row, self.positions // PAGE] * PAGE + self.positions % PAGE
        self.freq = rope.freqs(DIM)
        # two experts for each token, rows in the order of the experts
        expert = torch.stack([torch.randperm(COUNT, generator=g, device="cuda")[:2] for _ in range(T)]).flatten()
        order = torch.argsort(expert, stable=True)
        self.rows = (order // 2).contiguous()
        self.groups = torch.cat([torch.zeros(1, device="cuda"), torch.bincount(expert, minlength=COUNT).cumsum(0)]).to(torch.int32)
        self.back = torch.argsort(order).view(T, 2)

    def step(self):
        T = self.x.shape[0]
        s = {}
        s["codes1"], s["scales1"], s["res1"] = qg.rms_norm_fp8_b128(self.x, self.norms[0], self.residual)
        s["qkv"] = qg.qmm_fp8_b128(s["codes1"], s["scales1"], *self.qkv, out_dtype=torch.bfloat16)
        parts = s["qkv"].view(T, HEADS + 2 * KV_HEADS, DIM)
        s["q"] = qg.kv_append_rope(parts[:, :HEADS], parts[:, HEADS:HEADS + KV_HEADS], parts[:, HEADS + KV_HEADS:],
                                   self.positions, self.freq, *self.cache, self.slots)
        s["heads"] = qg.attn_paged(s["q"], *self.cache, self.table, self.offsets, self.context, max_new=max(self.new))
        s["attended"] = qg.qmm_fp8_b128(*qg.quantize_fp8_b128(s["heads"].view(T, HEADS * DIM)), *self.out,
                                        out_dtype=torch.bfloat16)
        s["codes2"], s["scales2"], s["res2"] = qg.rms_norm_fp8_b128(s["attended"], self.norms[1], s["res1"])
        s["codes3"], s["scales3"] = s["codes2"].view(torch.uint8)[self.rows].view(E4M3), s["scales2"][self.rows]
        s["wide"] = qg.qmm_fp8_b128_grouped(s["codes3"], s["scales3"], *self.up, self.groups, out_dtype=torch.bfloat16)
        s["codes4"], s["scales4"] = qg.silu_mul_fp8_b128(s["wide"][:, :WIDE], s["wide"][:, WIDE:])
        s["narrow"] = qg.qmm_fp8_b128_grouped(s["codes4"], s["scales4"], *self.down, self.groups)
        s["y"] = s["narrow"][self.back].sum(1)
        return s


def coded_is(codes, scales, y):
    want = qg.quantize_fp8_b128(y)
    assert torch.equal(codes.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scales, want[1])


def test_a_layer_step_by_step():
    m = Layer(1)
    old = [c.clone() for c in m.cache]
    s = m.step()
    T = m.x.shape[0]
    y1, r1 = qg.rms_norm(m.x, m.norms[0], m.residual, out_dtype=torch.float32)
    norms.check(y1, norms.ref(m.x, m.norms[0], m.residual, 1e-6, 0.0), HIDDEN)
    coded_is(s["codes1"], s["scales1"], y1)
    assert torch.equal(s["res1"], r1) and torch.equal(r1, m.x.float() + m.residual)
    check_product(s["qkv"], s["codes1"], s["scales1"], *m.qkv)
    parts = s["qkv"].view(T, -1, DIM)
    rope.check(s["q"], *rope.rotate(parts[:, :HEADS], m.positions, m.freq, False))
    rope.check(m.cache[0][m.slots // PAGE, :, m.slots % PAGE],
               *rope.rotate(parts[:, HEADS:HEADS + KV_HEADS], m.positions, m.freq, False))
    assert torch.equal(m.cache[1][m.slots // PAGE, :, m.slots % PAGE], parts[:, HEADS + KV_HEADS:])
    for c, o in zip(m.cache, old):
        o[m.slots // PAGE, :, m.slots % PAGE] = c[m.slots // PAGE, :, m.slots % PAGE]
        assert torch.equal(c, o)
    y2, r2 = qg.rms_norm(s["attended"], m.norms[1], s["res1"], out_dtype=torch.float32)
    norms.check(y2, norms.ref(s["attended"], m.norms[1], s["res1"], 1e-6, 0.0), HIDDEN)
    coded_is(s["codes2"], s["scales2"], y2)
    at = m.groups.tolist()
    assert at[-1] == 2 * T
    for e in range(COUNT):
        r = slice(at[e], at[e + 1])
        check_product(s["wide"][r], s["codes3"][r], s["scales3"][r], m.up[0][e], m.up[1][e])
        check_product(s["narrow"][r], s["codes4"][r], s["scales4"][r], m.down[0][e], m.down[1][e])
    gate = qg.silu_mul(s["wide"][:, :WIDE], s["wide"][:, WIDE:], out_dtype=torch.float32)
    gates.check(gate, s["wide"][:, :WIDE], s["wide"][:, WIDE:])
    coded_is(s["codes4"], s["scales4"], gate)
    assert qg.device_error() == 0


def same(a, b):
    return all(torch.equal(a[k].contiguous().view(torch.uint8), b[k].contiguous().view(torch.uint8)) for k in a)


def test_a_layer_in_graphs_beside_each_other():
    layers = [Layer(2), Layer(3)]
    want = [m.step() for m in layers]
    made = [captured(m.step) for m in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(10):
        for _, out in made:
            for v in out.values():
                v.view(torch.uint8).zero_()
        torch.cuda.synchronize()
        for s, (graph, _) in zip(streams, made):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(same(w, out) for w, (_, out) in zip(want, made))
    assert qg.device_error() == 0


def odd_experts(seed, counts):
    """Rows of 333 bytes: the calls copy them through scratch."""
    c = Experts(seed, counts, 130, 333)
    return c, c.run()


def test_threads_and_graphs_with_scratch():
    cases = [odd_experts(5, [3, 0, 40]), odd_experts(6, [200, 7, 150])]

    def work(i):
        torch.cuda.synchronize()
        return sum(not torch.equal(cases[i][0].run(), cases[i][1]) for _ in range(100))

    assert in_threads(work, 2) == [0, 0]
    made = [captured(c.run) for c, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (graph, out) in zip(streams, made):
            with torch.cuda.stream(s):
                out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for (_, out), (_, want) in zip(made, cases))
    assert qg.device_error() == 0


def test_first_call_of_a_thread():
    few, many = Experts(7, [3, 9], 256, 512), Experts(8, [300, 520], 256, 512)
    for c in (few, many):
        want = c.run()
        torch.cuda.synchronize()
        assert torch.equal(in_threads(lambda i: c.run(), 1)[0], want)


def test_on_a_given_stream():
    """Outputs and work of a call with a stream belong to it."""
    m = Layer(9)
    c = Experts(10, [5, 60, 0, 300], 200, 512)
    x = torch.randn(64, 2048, generator=rng(11), device="cuda")
    calls = [lambda s: qg.rms_norm(x, stream=s), lambda s: qg.silu_mul_fp8_b128(x, x, stream=s)[0].view(torch.uint8),
             lambda s: qg.qmm_fp8_b128_grouped(c.a, c.sa, c.w, c.sw, c.offsets, stream=s),
             lambda s: qg.kv_append_rope(x.view(64, 16, 128), x[:, :256].unflatten(1, (2, 128)), x[:, 256:512].unflatten(1, (2, 128)),
                                         torch.arange(64, device="cuda"), rope.freqs(128),
                                         *[torch.zeros(8, 2, 16, 128, device="cuda").half() for _ in range(2)],
                                         torch.arange(64, device="cuda"), stream=s)]
    assert same(m.step(), m.step())
    side = torch.cuda.Stream()
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        old = [torch.empty_like(want) for _ in range(6)]
        torch.cuda._sleep(20_000_000)
        for t in old:
            t.view(torch.uint8).fill_(7)
        del old, t
        side.wait_stream(torch.cuda.default_stream()) if call is calls[3] else None
        got = call(side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_rows_do_not_depend_on_the_batch():
    m = Layer(12)
    x = torch.randn(300, 1000, generator=rng(13), device="cuda").bfloat16()
    y, codes = qg.rms_norm(x), qg.silu_mul_fp8_b128(x, x)[0].view(torch.uint8)
    for i in (0, 7, 299):
        assert torch.equal(qg.rms_norm(x[i:i + 1])[0], y[i])
        assert torch.equal(qg.silu_mul_fp8_b128(x[i:i + 1], x[i:i + 1])[0].view(torch.uint8)[0], codes[i])
    q = torch.randn(700, 3, 64, generator=rng(14), device="cuda")
    positions, slots = torch.arange(700, device="cuda"), torch.full((700,), -1, device="cuda")
    all_rows = qg.kv_append_rope(q, q[:, :2], q[:, :2], positions, m.freq, *m.cache, slots)
    one = qg.kv_append_rope(q[333:334], q[333:334, :2], q[333:334, :2], positions[333:334], m.freq, *m.cache, slots[:1])
    assert torch.equal(all_rows[333], one[0])


@pytest.mark.parametrize("counts,N,K", [([0] * 1023 + [5], 40, 128), ([1] * 1024, 130, 256), ([0, 700] + [0] * 500, 130, 256),
                                        ([0] * 300 + [9000], 64, 128)])
def test_many_experts(counts, N, K):
    c = Experts(len(counts), counts, N, K)
    y = c.run(out_dtype=torch.bfloat16)
    c.check(y, [e for e, n in enumerate(counts) if n][:40])
    assert qg.device_error() == 0


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_independent_projection_after_each(pdl, mode):  # noqa: F811
    """A projection that has nothing to do with the call before it, but with what came before that."""
    n, k = 4096, 4096
    w = projection(30, n, k)
    g = rng(31)
    big = torch.randn(4096, 4096, generator=g, device="cuda")
    x = torch.empty(1, k, device="cuda")
    small = torch.randn(3, 5000, generator=g, device="cuda")
    m = Layer(32)
    few, many, odd = Experts(33, [3, 0, 2], 256, 512), Experts(34, [300, 100], 256, 512), Experts(35, [3, 2], 256, 333)
    v = torch.randn(31, 2, 64, generator=g, device="cuda")
    serving = [lambda: qg.rms_norm(small), lambda: qg.silu_mul(small, small), few.run, many.run, odd.run,
               lambda: qg.kv_append_rope(v, v, v, m.positions[:31], m.freq, *m.cache, m.slots[:31])]

    def run(mode):
        out = []
        for i, call in enumerate(serving):
            pdl(0)
            t = torch.full((4096, 1), 0.01 * (i + 1), device="cuda")
            for _ in range(3):
                t = torch.mm(big, t) / 64
            torch.mm(t.t(), big, out=x)  # (some time on the way, so that a call that does not wait reads the old x)
            call()
            pdl(mode)
            out.append(qg.qgemv_q4_k(w, x, N=n))
        return out

    want = run(0)
    for a, b in zip(want, run(mode)):
        assert torch.equal(a, b)
    assert qg.device_error() == 0


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_after_independent_projections(pdl, mode):  # noqa: F811
    """Projections that need not wait for each other, then a call that reads what all of them wrote."""
    n, parts = 4096, 3
    ws = [projection(40 + i, n, 4096) for i in range(parts)]
    g = rng(41)
    xs = [torch.randn(1, 4096, generator=g, device="cuda") for _ in range(8)]
    out = torch.empty(1, n * parts, device="cuda")
    pieces = [out[:, i * n:(i + 1) * n] for i in range(parts)]

    def step(x, mode):
        pdl(mode)
        for w, piece in zip(ws, pieces):
            qg.qgemv_q4_k(w, x, piece, N=n)
        y = qg.rms_norm(out)
        pdl(mode)
        for w, piece in zip(ws, pieces):
            qg.qgemv_q4_k(w, x, piece, N=n)
        return y, qg.silu_mul(out[:, :n], out[:, n:2 * n])

    want = [step(x, 0) for x in xs]
    got = [step(x, mode) for x in xs]
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert qg.device_error() == 0


def chain():
    """Layers one after the other, each fed by the one before, without a pause: the results of all of them."""
    m = Layer(50)
    out = []
    for _ in range(10):
        s = m.step()
        m.x, m.residual = s["y"].bfloat16(), s["res2"]
        out.append(s)
    torch.cuda.synchronize()
    return [{k: v.cpu() for k, v in s.items()} for s in out]


def test_overlapped_layers_give_the_same(pdl, tmp_path):  # noqa: F811
    """In a process where QG_OPT_PDL has never been 2, calls start while the one before ends; here they do not."""
    code = "import sys, torch; sys.path[:0] = ['tests', '.']; import test_gpu_layer_calls as t; torch.save(t.chain(), sys.argv[1])"
    r = subprocess.run([sys.executable, "-c", code, str(tmp_path / "out.pt")], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    pdl(2)
    pdl(0)
    for a, b in zip(torch.load(tmp_path / "out.pt"), chain(), strict=True):
        assert same(a, b)
    assert qg.device_error() == 0


def test_a_tensor_without_data_raises():
    """Tensors inside torch.vmap have no address: an error, after which the process goes on."""
    x = torch.ones(3, 4, 256, device="cuda")
    for call in (qg.rms_norm, qg.rms_norm_fp8_b128, lambda x: qg.silu_mul(x, x)):
        with pytest.raises(RuntimeError):
            torch.vmap(call)(x)
    assert (qg.rms_norm(x[0], eps=0.0) == 1).all() and qg.device_error() == 0


def test_wide_codes_and_scales():
    """Codes of every exponent and scales over twelve binary orders, as in the products' tests, through both kernels."""
    g = rng(60)
    for counts in ([1, 30, 2], [257, 40, 130]):
        c = Experts(61, counts, 384, 1024)
        c.a, c.sa = codes_like(g, *c.a.shape), scales_like(g, *c.sa.shape)
        c.check(c.run())


def test_first_calls_of_a_process_are_captured():
    """No call before the capture: what a kernel's first call sets up and asks for is allowed there."""
    code = """
import sys, torch
sys.path[:0] = ["tests", "."]
import bit_quantized_gemv_dequant_gb300 as qg
import test_gpu_layer_calls as t
m, few, many, odd = t.Layer(1), t.Experts(2, [3, 9], 256, 512), t.Experts(3, [300, 520], 256, 512), t.Experts(4, [3, 9], 40, 250)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = m.step(), few.run(), many.run(), odd.run()
graph.replay()
torch.cuda.synchronize()
got = {k: v.clone() for k, v in out[0].items()}, [v.clone() for v in out[1:]]
assert t.same(got[0], m.step()) and all(torch.equal(a, b) for a, b in zip(got[1], (few.run(), many.run(), odd.run())))
assert qg.device_error() == 0
print("done")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["done"], (r.returncode, r.stdout, r.stderr[-2000:])


@pytest.mark.parametrize("M,K", [(200001, 3), (70000, 8), (3, 300000), (1, 1000003)])
def test_tall_and_wide(M, K):
    x = torch.randn(M, K, generator=rng(70), device="cuda").bfloat16()
    w = torch.rand(K, generator=rng(71), device="cuda") + 0.5
    y, r = qg.rms_norm(x, w, x, out_dtype=torch.float32)
    norms.check(y, norms.ref(x, w, x, 1e-6, 0.0), K)
    assert torch.equal(r, x + x)
    coded_is(*qg.rms_norm_fp8_b128(x, w, x)[:2], y)
    y = qg.silu_mul(x, x, out_dtype=torch.float32)
    gates.check(y, x, x)
    coded_is(*qg.silu_mul_fp8_b128(x, x), y)


@pytest.mark.parametrize("T,Hq,Hkv,D", [(100003, 1, 1, 8), (2, 65535, 3, 8), (3, 1, 300, 48)])
def test_many_tokens_and_many_heads(T, Hq, Hkv, D):
    rope.Case(72, T, Hq, Hkv, D, 64, "bf16", "bf16").check()
    rope.Case(73, T, Hq, Hkv, D, 64, "f32", "f16", rot=D // 2).check(True)


@pytest.mark.parametrize("counts,N,K", [([40] * 1000 + [0] * 24, 1, 16), ([129] * 300, 257, 144), ([1] * 700, 3, 100), ([100003], 8, 16)])
def test_many_rows_and_narrow_weights(counts, N, K):
    c = Experts(74, counts, N, K, 1, 1)
    y = c.full("f32")
    c.run(y=y)
    c.check(y, list(range(0, len(counts), 37)))
    assert (y[0] == 7).all() and (y[-1] == 7).all() and qg.device_error() == 0
