"""Inputs and error bounds shared by the GPU tests of attention, the norm and the 8-bit checkpoints."""
from __future__ import annotations

import numpy as np
import torch

import oracle

U = 2.0 ** -8      # unit roundoff of bf16: half of its spacing over its value


def rng(*key):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence(entropy=11, spawn_key=key)))


def bf16(a) -> np.ndarray:
    """float64 values rounded to bf16."""
    return oracle.f32_from_bf16_bits(oracle.bf16_bits_from_f32(np.asarray(a, dtype=np.float32))).astype(np.float64)


def dev(a: np.ndarray, dtype=torch.bfloat16) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype).to("cuda:0")


def host(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def within(name: str, got, ref, bound) -> None:
    """|got - ref| <= bound, element by element; -inf and the like have to be equal."""
    got, ref = host(got) if isinstance(got, torch.Tensor) else got, np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine]), f"{name}: infinities differ"
    assert np.all(np.isfinite(got[fine])), f"{name}: not finite"
    over = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)) - bound, -1.0)
    i = np.unravel_index(int(over.argmax()), over.shape) if over.size else ()
    assert not over.size or over[i] <= 0, f"{name}: at {i} got {got[i]:.6g}, want {ref[i]:.6g}, {over[i]:.3g} past the bound"
