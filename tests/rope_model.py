"""Norm, rotation and store in 64 bits on the CPU, from the formulas."""
import numpy as np
import torch


def table(max_position, rot, base=10000.0):
    angle = np.arange(max_position)[:, None] * base ** (-np.arange(rot // 2) * 2.0 / rot)
    return torch.tensor(np.concatenate([np.cos(angle), np.sin(angle)], 1), dtype=torch.float32)


def turned(x, weight, cos_sin, positions, pair_axis, interleaved, eps):
    """[tokens, heads, D] float64 of bf16 inputs; positions [axes, tokens]."""
    x = x.double().cpu().numpy().copy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.double().cpu().numpy()
    cs = cos_sin.double().cpu().numpy()
    half = cs.shape[1] // 2
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        row = cs[np.asarray(positions)[pair_axis[i]]]
        c, s = row[:, i][:, None], row[:, half + i][:, None]
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, b] * c + x[:, :, a] * s
    return y
