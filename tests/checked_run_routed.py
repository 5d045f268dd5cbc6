"""Routed-field and distillation calls through the checked library: no failed
index check on valid plans, and a place outside the slots is recorded (and
skipped).  Run as a process of its own by test_gpu_zchecked_routed.py."""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import volume_rendering_amd as v  # noqa: E402
from volume_rendering_amd import _binding as B  # noqa: E402

B._LIB_PATH = os.path.join(ROOT, "volume_rendering_amd", "libnerf_mi355x_checked.so")


def check(what):
    torch.cuda.synchronize()
    f = B.nerf_check_flags()
    print(f"{what}: flags {f:#x}", flush=True)
    return f


def main():
    g = np.random.default_rng(3)
    bad = B.nerf_check_flags()
    i32 = dict(dtype=torch.int32, device="cuda")
    for n, k, E, d, o, dt in ((3, 2, 16, 96, 64, torch.bfloat16), (5000, 2, 8, 64, 136, torch.bfloat16),
                              (60000, 2, 5, 64, 264, torch.bfloat16), (9001, 1, 4096, 63, 32, torch.float32),
                              (2000, 3, 7, 130, 77, torch.float32)):
        ids = g.integers(-1, E, (n, k)).astype(np.int32)
        S = n * k
        off, order, place = torch.empty(E + 1, **i32), torch.empty(S, **i32), torch.empty((n, k), **i32)
        v.nerf_route_plan(torch.from_numpy(ids).cuda(), E, off, order, place)
        x = torch.randn((n, d), device="cuda").to(dt)
        rows, y = torch.empty((S, d), dtype=dt, device="cuda"), torch.empty((S, o), dtype=dt, device="cuda")
        w = torch.randn((E, o, d), device="cuda").to(dt)
        wt = torch.rand((n, k), device="cuda")
        v.nerf_route_gather(x, off, place, rows)
        v.nerf_expert_linear(x, w, None, off, y, order=order, k=k, relu=True)
        v.nerf_expert_linear(rows, w, None, off, y)
        out, dy, dw = torch.empty((n, o), dtype=dt, device="cuda"), torch.empty_like(y), torch.empty_like(wt)
        v.nerf_route_combine(y, off, place, wt, out)
        v.nerf_route_combine_grad(out, y, off, place, wt, dy, dw)
        gw, gb = torch.empty(w.shape, device="cuda"), torch.empty((E, o), device="cuda")
        v.nerf_expert_linear_grad(dy, x, w, off, rows, gw, gb, order=order, k=k, relu_x=True)
        v.nerf_expert_linear_grad(dy, rows, w, off, None, gw, gb)
        bad |= check(f"n={n} k={k} experts={E} {d}->{o}")
    if bad:
        print(f"FAILED: index checks recorded {bad:#x}")
        return 1
    # positive control: the last pair's place lies just outside the slots
    place[-1, -1] = S
    v.nerf_route_gather(x, off, place, rows)
    if check("positive control") != 1 << 9:
        print("FAILED: the control should set bit 9 alone")
        return 1
    print("checked library: no failed index check; the control was recorded")
    return 0


if __name__ == "__main__":
    sys.exit(main())
