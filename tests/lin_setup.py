"""Helpers of the norms' and projections' tests: handles, tensors, weights."""
import contextlib

import numpy as np
import torch

import fp4_block_scaled_gb300 as moe
from oracle import lin as ol

MODE = {"none": moe.MOE_ACT_BF16, "e4m3": moe.MOE_ACT_E4M3_UE8M0_128, "e2m1": moe.MOE_ACT_E2M1_UE8M0_32}
TYPE = {"bf16": moe.MOE_OUT_BF16, "f32": moe.MOE_OUT_F32}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@contextlib.contextmanager
def handle(max_tokens=0, max_in=0):
    h = moe.moe_lin_create(moe.lin_config(max_tokens, max_in), 0)
    try:
        yield h
    finally:
        torch.cuda.synchronize()
        moe.moe_lin_destroy(h)


def f64(t):
    return t.detach().double().cpu().numpy()


def code_buffers(rows, n, fmt, fill=0xEE):
    """Codes and scales of `rows` rows and one more, filled."""
    width, block = (n // 2, 32) if fmt == "e2m1" else (n, 128)
    return (torch.full((rows + 1, width), fill, dtype=torch.uint8, device="cuda"),
            torch.full((rows + 1, -(-n // block)), fill, dtype=torch.uint8, device="cuda"))


def rand(rng, shape, scale=1.0):
    return torch.from_numpy(scale * rng.standard_normal(shape)).float().cuda()


class Weights:
    """Random E2M1 weights of a linear layer, packed."""

    def __init__(self, h, N, K, rng, lo=117, hi=124):
        self.N, self.K = N, K
        self.codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
        self.scales = rng.integers(lo, hi, (N, K // 32), dtype=np.uint8)
        self.pack(h)

    def pack(self, h):
        self.dev = [torch.from_numpy(a).cuda() for a in (self.codes, self.scales)]
        self.packed = torch.full((moe.moe_linear_packed_bytes(self.N, self.K),), 0xFF, dtype=torch.uint8, device="cuda")
        moe.moe_linear_pack(h, *self.dev, self.N, self.K, self.packed)
        self.desc = moe.linear(self.packed, self.N, self.K)
        return self

    def values(self):
        return ol.values(self.codes, self.scales, "e2m1")
