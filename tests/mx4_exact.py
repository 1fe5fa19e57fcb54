"""Operands whose MXFP4 sums are exact in fp32, and their results in float64 on the GPU: a kernel that takes
every element once, in any order, returns the correctly rounded exact result bit for bit."""
import ctypes

import numpy as np
import torch

import nvfp4_block_scaled_02_amd as nv
from oracle import mxfp4_oracle as M4


def u8(shape, seed, lo=0, hi=256):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda", generator=g)


def values(packed, scales):
    """float64 values of device tensors of codes and scale bytes."""
    table = torch.tensor(np.concatenate([M4.E2M1_POS, -M4.E2M1_POS]), device=packed.device)
    v = table[torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2).long()]
    return v * torch.exp2(scales.double() - 127.0).repeat_interleave(32, dim=-1)


def guarded_u8(t):
    """A copy between bytes that read as NaN scales."""
    base = torch.full((t.numel() + 8192,), 0xFF, dtype=torch.uint8, device="cuda")
    view = base[4096: 4096 + t.numel()].view(t.shape)
    view.copy_(t)
    return view


def mxfp4_form(M, N, K):
    form, fused = (ctypes.c_int * 4)(), ctypes.c_int()
    assert nv.load_library().nvfp4_selftest_mxfp4_form(M, N, K, 0, form, ctypes.byref(fused)) == 0
    return tuple(form), bool(fused.value)


def moe_form(T, E, k, H, I):
    """(who routes, staged, few, whether the second product has shares)"""
    form = (ctypes.c_int * 4)()
    assert nv.load_library().nvfp4_selftest_moe_form(T, E, H, I, k, form) == 0
    return form[0], form[1], form[2], int(form[3] > 0)
