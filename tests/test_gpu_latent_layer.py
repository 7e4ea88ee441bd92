"""The example layer of latent attention: prompts in chunks through the expanded
form, then single tokens through the absorbed form in a replayed graph, against
the same layer in fp32.

With e4m3 latents, off by up to 2^-4 of themselves, evenly spread: 2^-4 /
sqrt(3) rms at most, 3.6 %; keys and values, sums over independent latents, are
off by as much of their rms, scores of unit size by as much of theirs, and a
softmax-weighted mean of values by the root of both squares, 5.1 %; held to 6 %.
With bf16 latents what remains are roundings to bf16, 2^-8 / sqrt(3) = 0.23 %
rms at most each, ten on the way of a value: 0.8 %, and as many on the way of a
score: 1.1 % together; held to 2 %."""

import importlib.util
import os

import pytest
import torch

from tests.test_gpu_latent import OwnStream

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("latent_layer", os.path.join(ROOT, "examples", "latent_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("heads,latent,lens,fmt,bound", [
    (8, 512, (300, 1, 130), "e4m3", 0.06), (8, 512, (300, 1, 130), "bf16", 0.02), (5, 256, (70,), "bf16", 0.02),
    (64, 256, tuple(range(3, 40, 2)), "e4m3", 0.06)])
def test_layer(gpu, example, monkeypatch, heads, latent, lens, fmt, bound):
    of_torch = torch.cuda.Stream
    monkeypatch.setattr(torch.cuda, "Stream", lambda **which: of_torch(**which) if which else OwnStream())
    print(f"[case] latent layer {heads} x {latent}, {len(lens)} prompts, {fmt}", flush=True)
    error, _ = example.serve(512, heads, latent, lens, steps=12, fmt=fmt, chunk=128)
    assert 0 < error < bound
