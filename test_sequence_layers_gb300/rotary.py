"""The cos / sin table that ``abi.ttt_rope`` reads, made once per model.

A pair i of the rot rotated features turns by pos * inv_i at position pos, inv_i =
base^(-2i/rot).  Long contexts stretch the frequencies:
  * "linear": positions divided by factor;
  * "ntk": the base raised by factor^(rot/(rot-2)), so that the slowest pair is divided
    by factor and the fastest keeps its frequency;
  * "yarn": by the number of turns a pair makes over the original context: beta_fast
    turns and more keep their frequency, beta_slow and fewer are divided by factor,
    linear between them; cos and sin carry the factor 0.1 ln(factor) + 1.
"""
from __future__ import annotations

import math

import torch


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_rows=8192, beta_fast=32.0,
                     beta_slow=1.0):
    """(inverse frequencies [rot/2] in fp64, factor on cos and sin)."""
    if rot < 0 or rot % 2:
        raise ValueError("rot must be even and not negative")
    if not factor > 0.0 or not base > 0.0:
        raise ValueError("base and factor must be positive")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    inv = base ** (-2.0 * i / max(rot, 1))
    if scaling in ("none", "ntk"):
        return inv, 1.0
    if scaling == "linear":
        return inv / factor, 1.0
    if scaling == "yarn":
        if not beta_fast > beta_slow:
            raise ValueError("beta_fast must exceed beta_slow")
        turns = original_rows * inv / (2.0 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        return inv * keep + inv / factor * (1.0 - keep), (0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0)
    raise ValueError('scaling must be "none", "linear", "ntk" or "yarn"')


def rope_table(rows, rot, device="cuda", **scaling):
    """fp32 [rows, rot/2, 2]: cos and sin at positions 0 .. rows-1, computed in fp64 and
    rounded once (an fp32 product of a large position with a frequency would lose its
    angle).  Keyword arguments as rope_frequencies."""
    inv, m = rope_frequencies(rot, **scaling)
    ang = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * inv.to(device)
    return (m * torch.stack([ang.cos(), ang.sin()], -1)).float().contiguous()


def rope_axes(sections, layout="blocks"):
    """The axis of every pair, for ``abi.ttt_rope_axes``: sections[a] pairs turn by axis a,
    one block after the other ("blocks") or the axes in turn for as long as each has pairs
    left ("cyclic")."""
    sections = [int(n) for n in sections]
    if not sections or min(sections) < 0:
        raise ValueError("sections must be the axes' numbers of pairs")
    if layout == "blocks":
        return bytes(a for a, n in enumerate(sections) for _ in range(n))
    if layout == "cyclic":
        return bytes(a for j in range(max(sections)) for a, n in enumerate(sections) if j < n)
    raise ValueError('layout must be "blocks" or "cyclic"')


def pair_bytes(axes):
    """A sequence of the pairs' axes, one byte each (a number is none: bytes(n) would be n zeros,
    and an array's bytes() its memory)."""
    try:
        return bytes([*axes])
    except TypeError:
        raise ValueError("pair_axis must be a sequence of integers") from None


def rope_axes_table(rows, pair_axis, per_axis=True, device="cuda", **scaling):
    """The table of ``abi.ttt_rope_axes``, fp32 [rows, rot/2, 2].  per_axis: every axis has
    the frequencies of a head of its own pairs alone (a picture's two halves); else pair i
    keeps the frequency it has with one axis.  Keyword arguments as rope_frequencies, per
    axis if per_axis."""
    pair_axis = pair_bytes(pair_axis)
    inv, m = rope_frequencies(2 * len(pair_axis), **scaling)
    if per_axis:
        for a in set(pair_axis):
            at = [i for i, b in enumerate(pair_axis) if b == a]
            inv[at], m = rope_frequencies(2 * len(at), **scaling)
    ang = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * inv.to(device)
    return (m * torch.stack([ang.cos(), ang.sin()], -1)).float().contiguous()
