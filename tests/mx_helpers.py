"""Helpers of the microscaled operators' tests: device matrices from the 64-bit
oracle's codes and back."""
import numpy as np
import torch

import lora_adapter_application_b200 as lora
from oracle import mx


def to_device(codes, scales, fmt, cols, device="cuda"):
    """An MxTensor of the oracle's codes [rows, padded] and scale bytes."""
    rows = codes.shape[0]
    return lora.MxTensor(rows, cols, fmt,
                         q=torch.from_numpy(np.ascontiguousarray(mx.pack(codes, fmt))).to(device),
                         scales=torch.from_numpy(mx.pack_scales(scales)).to(device))


def from_device(m):
    """(codes, scale bytes) of an MxTensor."""
    return (mx.unpack(m.q.cpu().numpy().reshape(m.rows, -1), m.fmt),
            mx.unpack_scales(m.scales.cpu().numpy(), m.rows, m.cols))


def as64(t):
    return t.detach().cpu().double().numpy()
