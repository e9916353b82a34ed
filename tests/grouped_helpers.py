"""Inputs and bounds of the grouped-product tests."""
import numpy as np
import torch

DEV = "cuda:0"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}

# queue lengths: none at all, one row, around the tile edges, empty queues
# first, between and last, one long queue beside many short ones
QUEUES = {
    "one row": [1],
    "all empty": [0, 0, 0],
    "edges": [0, 1, 31, 32, 33, 0, 63, 64, 65, 0],
    "long": [0, 127, 128, 129, 0, 255, 256, 257, 3],
    "skewed": [700, 1, 0, 2, 1, 0, 0, 5],
    "decode 256": [1 if e % 3 == 0 else 0 for e in range(256)],
    "dense": [333],
}


def offsets_of(counts, start=0):
    return np.concatenate([[start], start + np.cumsum(counts)]).astype(np.int32)


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(seed, *shape, dtype="bf16", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(TORCH[dtype])


def check(got, ref, terms, length, dtype, what=""):
    """|got - ref| against the bound of a float32 accumulation of ``length``
    terms and one rounding to ``dtype``: every product and partial sum is
    rounded at most once on its way (in any order), (length + 1) 2^-24 times
    the sum of the terms' absolute values, doubled for a matrix unit that
    truncates; then half a step of the output type.  Rows whose reference is
    NaN are not compared."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape
    have = ~np.isnan(ref)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    bound = 2.0 * (length + 1) * 2.0 ** -24 * terms + half * np.abs(ref) * (1 + 2.0 ** -8) + 2.0 ** -126
    err = np.abs(got - ref)
    bad = have & ~(err <= bound)
    if bad.any():
        at = np.argwhere(bad)[0]
        raise AssertionError(f"{what}: {bad.sum()} of {have.sum()} out of bounds, first at {tuple(at)}: "
                             f"{got[tuple(at)]} for {ref[tuple(at)]}, bound {bound[tuple(at)]}")
