"""Streaming-field calls through the checked library: no failed index check on
valid offsets, and an offset past the rows is recorded (and kept in range).  Run
as a process of its own by test_gpu_zchecked_streaming.py."""
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
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    for n, E, k, d, h, o, dt in ((1, 16, 2, 96, 64, 40, bf), (40, 3, 2, 63, 33, 9, f32), (100, 4, 5, 130, 70, 40, bf)):
        z = torch.randn((n, E), device="cuda").to(dt)
        ids, w = torch.empty((n, min(k, E)), dtype=i32, device="cuda"), torch.empty((n, min(k, E)), device="cuda")
        v.nerf_route_gate(z, ids, w)
        v.nerf_route_gate_grad(torch.randn_like(w), z, ids, w, torch.empty_like(z), renorm=False)
        x, out = torch.randn((n, d), device="cuda").to(dt), torch.empty((n, o), dtype=dt, device="cuda")
        w1, w2 = torch.randn((E, h, d), device="cuda").to(dt), torch.randn((E, o, h), device="cuda").to(dt)
        v.nerf_routed_mlp(x, ids, w, w1, None, w2, None, out)
        bad |= check(f"gate and layer n={n} k={k} experts={E} {d}->{h}->{o}")
    for lens, d, gates, dt in (([1, 0, 70, 9], 24, 3, f32), ([5000, 0, 300], 70, 70, bf), ([60] * 40, 600, 1, bf)):
        off = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
        rows = int(off[-1])
        a, x = torch.rand((rows, gates), device="cuda"), torch.randn((rows, d), device="cuda").to(dt)
        hh, h0 = torch.empty_like(x), torch.randn((len(lens), d), device="cuda")
        v.nerf_scan(a, x, hh, h0=h0, offsets=off, mix=True)
        v.nerf_scan_grad(x, a, x, hh, torch.empty_like(a), torch.empty_like(x), h0=h0, offsets=off, mix=True)
        bad |= check(f"recurrence of {rows} rows d={d} gates={gates}")
    grads = [torch.randn(int(s), device="cuda").to((f32, bf)[i % 2]) for i, s in enumerate(g.integers(0, 40000, 90))]
    v.nerf_grad_clip(v.nerf_tensor_list(grads), 1.0, torch.empty(1, device="cuda"))
    bad |= check("90 gradients")
    if bad:
        print(f"FAILED: index checks recorded {bad:#x}")
        return 1
    # positive control: the last sequence ends one row past the rows
    off[-1] += 1
    v.nerf_scan(a, x, hh, offsets=off)
    if check("positive control") != 1 << 11:
        print("FAILED: the control should set bit 11 alone")
        return 1
    print("checked library: no failed index check; the control was recorded")
    return 0


if __name__ == "__main__":
    sys.exit(main())
