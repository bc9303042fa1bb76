"""The serving example: the same tokens, batched, chunked and continued in different ways, have the same log
probabilities. Keys, values and outputs are rounded to bf16 (2^-8) and activations to e4m3 (2^-4 of a value, or of a
neighbouring one after a different rounding before it) in two layers; probabilities of 1 / 1024 then move by some
hundredths, and an error in a page or an offset moves them by ones."""
import importlib.util
import os

import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg
from conftest import ROOT

pytestmark = pytest.mark.gpu


def test_the_ways_agree():
    spec = importlib.util.spec_from_file_location("serving_step", os.path.join(ROOT, "examples", "serving_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    far = example.main()
    assert set(far) == {"prompts together", "token by token", "continuations", "after packing"}
    for what, value in far.items():
        assert value < 0.1, (what, value)


def test_outputs_on_a_given_stream_are_apart_from_work_under_way():
    """Memory given back while the current stream still writes to it is not an output on another stream."""
    x = torch.randn(64, 4096, device="cuda")
    want = qg.quantize_fp8_b128(x)
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        old = [torch.empty_like(t) for t in want for _ in range(4)]
        torch.cuda._sleep(20_000_000)
        for t in old:
            t.view(torch.uint8).fill_(7)
        del old, t
        got = qg.quantize_fp8_b128(x, stream=side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_captured_call_keeps_its_scratch():
    """A graph replayed after the stream's scratch has grown."""
    g = torch.Generator("cuda").manual_seed(1)
    w, sw = torch.randn(256, 520, generator=g, device="cuda").to(torch.float8_e4m3fn)[:, :519].contiguous(), torch.rand(
        2, 5, generator=g, device="cuda")
    a, sa = qg.quantize_fp8_b128(torch.randn(40, 519, generator=g, device="cuda"))
    want = qg.qmm_fp8_b128(a, sa, w, sw)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        qg.qmm_fp8_b128(a, sa, w, sw)
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            y = qg.qmm_fp8_b128(a, sa, w, sw)
        big, sbig = qg.quantize_fp8_b128(torch.randn(9000, 519, generator=g, device="cuda"))
        qg.qmm_fp8_b128(big, sbig, w, sw)
        hold = [torch.full((1 << 18,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(40)]
        graph.replay()
    torch.cuda.synchronize()
    assert len(hold) == 40 and torch.equal(y, want)
    assert qg.device_error() == 0
