"""Run the grouping and lora_add_linear a few times on one synthetic workload
layer, for profilers (ncu, nsys) or a quick check on a new device.

    python -m lora_adapter_application_b200.run_case prefill --reps 3 --requests 16
    python -m lora_adapter_application_b200.run_case decode_qproj --min-run 0
    python -m lora_adapter_application_b200.run_case decode_qproj --base mxfp8   # norm and 4-bit base product first
    python -m lora_adapter_application_b200.run_case decode_qproj --base bf16    # norm and dense base product first
    python -m lora_adapter_application_b200.run_case decode_qproj --experts 8    # and a block of 8 experts on the rows

Prints the tile counts and the device status word; exits non-zero on a
non-zero status.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import lora_adapter_application_b200 as lora  # noqa: E402
import workloads  # noqa: E402


class Base:
    """The layer's norm and its base product, weights in MXFP4 and rows in ``fmt``, or both dense (``fmt`` None), random:
    what fills y before the adapters' delta."""

    def __init__(self, x, y, fmt, status):
        (T, d), n = x.shape, y.shape[1]
        self.x, self.y, self.status = x, y, status
        self.residual, self.h = torch.zeros_like(x), torch.empty_like(x)
        self.sum = torch.empty_like(x)
        self.weight = torch.ones(d, dtype=x.dtype, device=x.device)
        self.q, self.w = None, torch.randn(n, d, device=x.device, dtype=x.dtype) / d ** 0.5
        if fmt is not None:
            dense = self.w
            self.q, self.w = lora.MxTensor(T, d, fmt), lora.MxTensor(n, d, lora.LORA_MXFP4)
            lora.lora_mx_quantize(self.w, dense)

    def step(self):
        """The normalised rows, which the adapters read too."""
        lora.lora_rms_norm(self.h, self.x, self.weight, 1e-5, residual=self.residual, residual_out=self.sum, q=self.q)
        if self.q is None:
            lora.lora_linear(self.y, self.h, self.w, self.status)
        else:
            lora.lora_mx_linear(self.y, self.q, self.w, self.status)
        return self.h


class Experts:
    """A feed-forward block of N experts (random, d -> 2 f -> d) over the layer's rows: two of them a row."""

    def __init__(self, x, N, f, status):
        T, d = x.shape
        self.k, self.N, self.status = min(2, N), N, status
        new = lambda *s: torch.randn(*s, device=x.device, dtype=x.dtype) / s[-1] ** 0.5   # noqa: E731
        self.router, self.up, self.down = new(N, d), new(N, 2 * f, d), new(N, d, f)
        self.logits = torch.empty(T, N, device=x.device, dtype=x.dtype)
        self.ids = torch.empty(T, self.k, dtype=torch.int32, device=x.device)
        self.weights = torch.empty(T, self.k, device=x.device)
        self.meta = lora.Meta(T * self.k, N, min_run=0, device=x.device)
        self.h = torch.zeros(T * self.k, f, device=x.device, dtype=x.dtype)
        self.z = torch.zeros(T * self.k, d, device=x.device, dtype=x.dtype)
        self.y = torch.empty_like(x)

    def step(self, x):
        lora.lora_linear(self.logits, x, self.router, self.status)
        lora.lora_expert_route(self.ids, self.weights, self.logits)
        lora.lora_build_segments(self.ids.view(-1), self.meta, self.status)
        lora.lora_expert_linear(self.h, x, self.up, self.meta, self.status, x_div=self.k, act=lora.ACT_SILU, gated=True)
        lora.lora_expert_linear(self.z, self.h, self.down, self.meta, self.status)
        lora.lora_expert_sum(self.y, self.z, self.ids, self.weights, self.N, residual=x)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("workload", choices=sorted(workloads.NAMES))
    ap.add_argument("--layer", type=int, default=0)
    ap.add_argument("--reps", type=int, default=3)
    ap.add_argument("--min-run", type=int, default=64, help="shortest run that becomes contiguous tiles (0 = none)")
    ap.add_argument("--rows-per-tile", type=int, default=lora.MAX_TILE_ROWS,
                    help="rows per gathered tile (1 .. 64)")
    ap.add_argument("--requests", type=int, default=0, help="prefill / mixed_70b: number of prompts (0 = default)")
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--base", choices=["none", "mxfp8", "mxfp4", "bf16"], default="none",
                    help="run the norm and the base product ahead of the adapters: rows in this format over weights in "
                         "MXFP4, or dense (bf16: the layer's own type)")
    ap.add_argument("--experts", type=int, default=0, help="run a block of so many experts over the layer's rows behind it")
    args = ap.parse_args(argv)

    kw = {"n_req": args.requests} if args.requests and args.workload in ("prefill", "mixed_70b") else {}
    w = workloads.make(args.workload, seed=args.seed, **kw)
    lay = w.layers[args.layer]
    dev = torch.device("cuda")
    x, y = lay.x.to(dev), lay.y0.to(dev)
    A, B = [a.to(dev) for a in lay.A], [b.to(dev) for b in lay.B]
    ids, ranks = w.ids.to(dev), w.ranks.to(dev)
    alphas = lora.alphas_full(w.alpha, w.N, dev)
    meta = lora.Meta(w.T, w.N, args.rows_per_tile, args.min_run, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    lora.lora_build_segments(ids, meta, status)
    base = None
    if args.base != "none":
        base = Base(x, y, {"mxfp8": lora.LORA_MXFP8, "mxfp4": lora.LORA_MXFP4, "bf16": None}[args.base], status)
    experts = Experts(x, args.experts, x.shape[1] // 2, status) if args.experts else None
    for _ in range(args.reps):
        if base is not None:
            x = base.step()
        lora.lora_add_linear(y, x, A, B, lay.col_off, ranks, alphas, meta, status)
        if experts is not None:
            experts.step(x)
    torch.cuda.synchronize()
    code = int(status.item())
    print(f"{w.name}/{lay.name}: T={w.T} counts={meta.counts.cpu().tolist()} status={code}")
    return 0 if code == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
