"""The operators of a streaming routed field, as measured.

Four operators:

``gate``   each sample's k largest of E gate logits and their softmax weights
           (``forward``); the logits' gradient (``backward``).
``layer``  the whole two-layer routed field for a few samples: every sample
           through its k experts, weighted and summed.
``scan``   the gated linear recurrence h_t = a_t h_{t-1} + b_t along packed
           sequences, b_t = x_t or (1 - a_t) x_t (``forward``), its gradients
           (``backward``), and one step of many states (sequences of length 1).
``clip``   the norm of all gradients of a list of tensors, and the gradients
           scaled down to a largest norm.

``run`` computes them in plain torch (float32, rounded once at the end), or
with this repository's entry points where ``own`` is true.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


def listed():
    gate = dict(op="gate", mask=0.0)
    layer = dict(op="layer", drop=0.0)
    scan = dict(op="scan", reverse=False, mix=False, state=True)
    return [
        # a training batch of 4096 rays x 64 samples, two of sixteen fields per sample
        dict(gate, name="gate_field", dir="forward", dtype="bf16", n=262144, experts=16, k=2, renorm=True),
        # gradients through the probabilities over all experts; odd sizes, some experts switched off for a sample
        dict(gate, name="gate_ragged_back", dir="backward", dtype="f32", n=20011, experts=61, k=3, renorm=False,
             mask=0.1),
        # one sample through two of sixteen experts: serving, latency and the weights of two experts
        dict(layer, name="layer_token", dtype="bf16", n=1, k=2, experts=16, d_in=1024, hidden=4096, d_out=1024,
             act="relu"),
        # the samples of one ray in a scene of one tiny network per cell, a third of them in empty space
        dict(layer, name="layer_cells", dtype="f32", n=64, k=1, experts=4096, d_in=63, hidden=32, d_out=4, act="relu",
             drop=0.3),
        # sixteen streams served together, four of 64 gated experts each: bound by the weights of the experts touched
        dict(layer, name="layer_streams", dtype="bf16", n=16, k=4, experts=64, d_in=1024, hidden=1024, d_out=1024,
             act="gated"),
        # two long sequences, a gate per channel kept in float32: training
        dict(scan, name="scan_long", dir="forward", dtype="bf16", gate_dtype="f32", n=2, len=32768, ragged=False,
             d=1024, gates=1024),
        dict(scan, name="scan_long_back", dir="backward", dtype="bf16", gate_dtype="f32", n=2, len=32768,
             ragged=False, d=1024, gates=1024),
        # features of 16 channels composited back to front along rays of 0 to 128 samples (empty space skipped)
        dict(scan, name="scan_rays", dir="forward", dtype="f32", gate_dtype="f32", n=65536, len=64, ragged=True, d=16,
             gates=1, reverse=True, mix=True, state=False),
        # a training batch's 256-wide features composited: one gate's gradient is a sum over all channels
        dict(scan, name="scan_rays_back", dir="backward", dtype="bf16", gate_dtype="bf16", n=4096, len=64, ragged=True,
             d=256, gates=1, reverse=True, mix=True, state=False),
        # one new sample for each of 256 streams: the state goes on by one step
        dict(scan, name="scan_step", dir="forward", dtype="bf16", gate_dtype="f32", n=256, len=1, ragged=False, d=1024,
             gates=1024, mix=True),
        # the parameter gradients of two 8 x 256 networks
        dict(op="clip", name="clip_nerf", shapes="nerf", copies=2, count=24, dtype="f32", max_norm=1.0),
        # two expert layers of sixteen 1024 -> 4096 experts, norms and biases between them
        dict(op="clip", name="clip_experts", shapes="experts", copies=1, count=32, dtype="both", max_norm=1.0),
    ]


# (rows, columns) of the weights of an 8 x 256 network with a skip, density, feature and colour heads; biases follow
_NERF = [(256, 63)] + [(256, 256)] * 4 + [(256, 319)] + [(256, 256)] * 2 + [(1, 256), (256, 256), (128, 283), (3, 128)]


def _sizes(case):
    """[(elements, type)] of a list of gradients."""
    if case["shapes"] == "nerf":
        one = [s for r, c in _NERF for s in (r * c, r)]
        return [(s, "f32") for s in one * case["copies"]]
    if case["shapes"] == "experts":
        one = [(16 * 4096 * 1024, "f32"), (16 * 4096, "f32"), (16 * 1024 * 4096, "bf16"), (16 * 1024, "f32")]
        small = [(1024, "f32"), (1024 * 16, "bf16"), (333, "f32"), (1, "f32")]
        return one + small * 7
    # sizes spread over a factor of `spread`, odd ones among them, in an order that mixes them
    out = []
    for i in range(case["count"]):
        u = (i * 7919 % case["count"]) / max(1, case["count"] - 1)
        size = max(1, int(case["largest"] * case["spread"] ** (u - 1.0)))
        out.append((size, case["dtype"] if case["dtype"] != "both" else ("f32", "bf16")[i % 2]))
    return out


def _lengths(case):
    """Sequence lengths: all alike, or evenly spread over 0 .. 2 len."""
    n, L = case["n"], case["len"]
    if not case["ragged"] or n == 1:
        return [L] * n
    return [i * (2 * L + 1) // n for i in range(n)]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 5e12, w["flops"] / 1e14)


def draw(rng):
    cap = {}
    for c in listed():
        cap[c["op"]] = max(cap.get(c["op"], 0.0), _cost(c))
    while True:
        op = rng.choice(["gate", "layer", "layer", "scan", "scan", "clip"])
        dtype = rng.choice(["f32", "bf16"])
        if op == "gate":
            c = dict(op=op, dir=rng.choice(["forward", "backward"]), dtype=dtype, n=_log_int(rng, 1, 262144),
                     experts=_log_int(rng, 2, 4096), k=rng.randint(1, 8), renorm=rng.choice([False, True]),
                     mask=rng.choice([0.0, 0.0, 0.1, 0.5]))
            c["k"] = min(c["k"], c["experts"])
        elif op == "layer":
            c = dict(op=op, dtype=dtype, n=_log_int(rng, 1, 128), k=rng.randint(1, 8), experts=_log_int(rng, 1, 4096),
                     d_in=_log_int(rng, 16, 4096), hidden=_log_int(rng, 16, 4096), d_out=_log_int(rng, 4, 4096),
                     act=rng.choice(["none", "relu", "gated"]), drop=rng.choice([0.0, 0.0, 0.1, 0.5]))
            c["k"] = min(c["k"], c["experts"])
            if rng.random() < 0.5:  # round widths as often as odd ones
                for key in ("d_in", "hidden", "d_out"):
                    c[key] = c[key] + 31 & ~31
            if c["n"] * c["k"] > 512 or c["experts"] * (c["d_in"] * 2 + c["d_out"]) * c["hidden"] > 1 << 28:
                continue
        elif op == "scan":
            c = dict(op=op, dir=rng.choice(["forward", "backward"]), dtype=dtype,
                     gate_dtype="f32" if dtype == "f32" else rng.choice(["f32", "bf16"]), n=_log_int(rng, 1, 65536),
                     len=_log_int(rng, 1, 65536), ragged=rng.choice([False, True]), d=_log_int(rng, 1, 2048),
                     reverse=rng.choice([False, True]), mix=rng.choice([False, True]),
                     state=rng.choice([False, True]))
            if rng.random() < 0.5:
                c["d"] = c["d"] + 31 & ~31
            divisors = [g for g in range(1, c["d"] + 1) if c["d"] % g == 0]
            c["gates"] = rng.choice([c["d"], c["d"], 1, rng.choice(divisors)])
            if c["n"] * c["len"] * c["d"] > 1 << 26:
                continue
        else:
            c = dict(op=op, shapes="spread", copies=1, count=_log_int(rng, 1, 400), dtype=rng.choice(["f32", "bf16", "both"]),
                     largest=_log_int(rng, 1, 1 << 26), max_norm=rng.choice([0.1, 1.0, 1e9]))
            c["spread"] = min(c["largest"], _log_int(rng, 1, 1 << 20))
        if _cost(c) <= cap[op]:
            return c


def work(case):
    if case["op"] == "gate":
        b, n, E, k = _SIZE[case["dtype"]], case["n"], case["experts"], case["k"]
        if case["dir"] == "forward":
            return {"bytes": n * E * b + 8 * n * k, "flops": 4 * n * E}
        reads = 12 * n * k + (0 if case["renorm"] else n * E * b)
        return {"bytes": reads + n * E * b, "flops": 4 * n * E}
    if case["op"] == "layer":
        b, pairs = _SIZE[case["dtype"]], case["n"] * case["k"] * (1 - case["drop"])
        E = case["experts"]
        touched = E * (1.0 - (1.0 - 1.0 / E) ** pairs) if E > 1 else 1.0
        up = 2 if case["act"] == "gated" else 1
        each = case["d_in"] * case["hidden"] * up + case["hidden"] * case["d_out"]
        bias = case["hidden"] * up + case["d_out"]
        return {"bytes": touched * (each * b + bias * 4) + case["n"] * (case["d_in"] + case["d_out"]) * b
                + 8 * case["n"] * case["k"], "flops": 2 * pairs * each}
    if case["op"] == "scan":
        b, ba, d, g = _SIZE[case["dtype"]], _SIZE[case["gate_dtype"]], case["d"], case["gates"]
        rows = sum(_lengths(case))
        state = 4 * case["n"] * d
        if case["dir"] == "forward":
            return {"bytes": rows * (2 * d * b + g * ba) + state * (1 + case["state"]), "flops": 2 * rows * d}
        streams = 4 if case["mix"] else 3  # dh, h, dx, and x
        return {"bytes": rows * (streams * d * b + 2 * g * ba) + state * 3 * case["state"], "flops": 4 * rows * d}
    byt = sum(s * _SIZE[t] for s, t in _sizes(case))
    return {"bytes": 2 * byt, "flops": 3 * sum(s for s, _ in _sizes(case))}


def _expert_ids(case, gen):
    """[n, k] int32: distinct experts per sample, uneven loads, -1 for a pair without an expert."""
    n, k, E = case["n"], case["k"], case["experts"]
    p = (torch.argsort(torch.rand(E, generator=gen, device="cuda")).float() + 1.0) ** (-0.5 if E <= 64 else -0.1)
    first = torch.multinomial(p, n, replacement=True, generator=gen)
    if k > 1:
        step = torch.randint(1, (E - 1) // (k - 1) + 1, (n, k - 1), generator=gen, device="cuda")
        ids = (first[:, None] + torch.cat([torch.zeros_like(step[:, :1]), step.cumsum(1)], 1)) % E
    else:
        ids = first[:, None]
    if case["drop"]:
        ids = torch.where(torch.rand(n, k, generator=gen, device="cuda") < case["drop"], -1, ids)
    return ids.to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    f32 = torch.float32

    def normal(*shape, scale=1.0, dtype=f32):
        return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    def empty(*shape, dtype=f32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    if own:
        import volume_rendering_amd as v
    s = dict(case=case)
    if case["op"] == "gate":
        n, E, k, dt = case["n"], case["experts"], case["k"], _DT[case["dtype"]]
        s["logits"] = normal(n, E, scale=2.0, dtype=dt)
        if case["mask"]:
            off = torch.rand(n, E, generator=gen, device="cuda") < case["mask"]
            s["logits"].masked_fill_(off, -math.inf)
        if case["dir"] == "backward":
            s["ids"], s["weights"] = _plain_gate(s["logits"], k, case["renorm"])
            s["dweights"] = normal(n, k)
        if own:
            if case["dir"] == "forward":
                s["out"] = (empty(n, k, dtype=torch.int32), empty(n, k))
            else:
                s["dlogits"] = empty(n, E, dtype=dt)
        return s
    if case["op"] == "layer":
        n, k, E, dt = case["n"], case["k"], case["experts"], _DT[case["dtype"]]
        din, hid, dout = case["d_in"], case["hidden"], case["d_out"]
        up = 2 * hid if case["act"] == "gated" else hid
        s["ids"] = _expert_ids(case, gen)
        s["weights"] = torch.rand(n, k, generator=gen, device="cuda").add_(0.05)
        s["weights"] /= s["weights"].sum(1, keepdim=True)
        s["x"] = normal(n, din, dtype=dt)
        s["w1"], s["b1"] = normal(E, up, din, scale=math.sqrt(2.0 / din), dtype=dt), normal(E, up, scale=0.1)
        s["w2"], s["b2"] = normal(E, dout, hid, scale=math.sqrt(2.0 / hid), dtype=dt), normal(E, dout, scale=0.1)
        if own:
            s["out"] = empty(n, dout, dtype=dt)
            s["ws"] = empty(max(1, v.nerf_routed_mlp_workspace_size(n, k, hid, dout)), dtype=torch.uint8)
        return s
    if case["op"] == "scan":
        dt, da, d, g, n = _DT[case["dtype"]], _DT[case["gate_dtype"]], case["d"], case["gates"], case["n"]
        lengths = torch.tensor(_lengths(case), dtype=torch.int64, device="cuda")
        lengths = lengths[torch.randperm(n, generator=gen, device="cuda")]
        s["offsets"] = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)]).to(torch.int32)
        rows = int(s["offsets"][-1])
        s["longest"] = int(lengths.max())
        # gates between 0 and 1, most of them near 1: states last for tens to thousands of steps
        s["a"] = torch.sigmoid(normal(rows, g, scale=1.5).add_(3.0)).to(da)
        s["x"] = normal(rows, d, dtype=dt)
        s["h0"] = normal(n, d) if case["state"] else None
        if case["dir"] == "backward":
            s["h"] = normal(rows, d, dtype=dt)  # (the states that a forward pass has left: any values)
            s["dh"] = normal(rows, d, dtype=dt)
            s["dh_last"] = normal(n, d) if case["state"] else None
        if own:
            kw = dict(gates=g, n_seq=n, backward=case["dir"] == "backward")
            s["ws"] = empty(max(1, v.nerf_scan_workspace_size(rows, d, **kw)), dtype=torch.uint8)
            if case["dir"] == "forward":
                s["h"], s["h_last"] = empty(rows, d, dtype=dt), empty(n, d)
            else:
                s["da"], s["dx"] = empty(rows, g, dtype=da), empty(rows, d, dtype=dt)
                s["dh0"] = empty(n, d) if case["state"] else None
        return s
    s["grads"] = [normal(size, scale=10.0 ** (i % 5 - 3), dtype=_DT[t]) for i, (size, t) in enumerate(_sizes(case))]
    if own:  # each tensor's place in one bucket for its type
        s["flat"] = {t: empty(sum(z for z, u in _sizes(case) if u == t), dtype=_DT[t]) for t in ("f32", "bf16")}
        at, outs = {"f32": 0, "bf16": 0}, []
        for size, t in _sizes(case):
            outs.append(s["flat"][t][at[t]:at[t] + size])
            at[t] += size
        s["list"] = v.nerf_tensor_list(s["grads"], outs)
        s["norm"] = empty(1)
        s["ws"] = empty(max(1, v.nerf_grad_norm_workspace_size(s["list"])), dtype=torch.uint8)
    return s


def _plain_gate(logits, k, renorm):
    z = logits.float()
    top, ids = torch.sort(z, dim=1, descending=True, stable=True)  # ties: the lowest index first
    top, ids = top[:, :k], ids[:, :k]
    m = top[:, :1].clamp_min(-3e38)  # (a row without an expert)
    e = (top - m).exp()
    total = (e if renorm else (z - m).exp()).sum(1, keepdim=True)
    weights = torch.where(total > 0, e / total, 0)
    ids = torch.where(top == -math.inf, -1, ids)
    return ids.to(torch.int32), weights


def _plain_gate_back(s, renorm):
    live = s["ids"] >= 0
    ids = s["ids"].clamp_min(0).long()
    wd = torch.where(live, s["weights"] * s["dweights"], 0)
    total = wd.sum(1, keepdim=True)
    z = s["logits"].float()
    if renorm:
        return torch.zeros_like(z).scatter_add_(1, ids, wd - torch.where(live, s["weights"], 0) * total).to(
            s["logits"].dtype)
    m = z.amax(1, keepdim=True).clamp_min(-3e38)
    e = (z - m).exp()
    norm = e.sum(1, keepdim=True)
    p = torch.where(norm > 0, e / norm, 0)
    return (-p * total).scatter_add_(1, ids, wd).to(s["logits"].dtype)


def _plain_layer(s):
    c = s["case"]
    n, k, hid = c["n"], c["k"], c["hidden"]
    ids = s["ids"].reshape(-1)
    e = ids.clamp_min(0).long()
    x = s["x"].float().repeat_interleave(k, 0)
    step = max(1, (1 << 28) // (hid * max(2 * c["d_in"], c["d_out"])))
    y = []
    for a in range(0, n * k, step):  # the experts' weights, gathered for a few pairs at a time
        ea = e[a:a + step]
        z = torch.bmm(s["w1"][ea].float(), x[a:a + step, :, None])[..., 0] + s["b1"][ea]
        if c["act"] == "gated":
            z = z[:, :hid] / (1.0 + (-z[:, :hid]).exp()) * z[:, hid:]
        elif c["act"] == "relu":
            z = z.clamp_min(0.0)
        y.append(torch.bmm(s["w2"][ea].float(), z[..., None])[..., 0] + s["b2"][ea])
    w = torch.where(ids >= 0, s["weights"].reshape(-1), 0)
    return (torch.cat(y) * w[:, None]).view(n, k, -1).sum(1).to(s["x"].dtype)


def _places(s, reverse):
    """[n, longest] rows in the order of the recurrence (or against it), and which of them exist."""
    off = s["offsets"].long()
    i = torch.arange(s["longest"], device="cuda")
    lo, hi = off[:-1, None], off[1:, None]
    rows = hi - 1 - i if reverse else lo + i
    return rows.clamp(0, int(s["x"].shape[0]) - 1), i < hi - lo


def _doubling(A, B):
    """B_t + A_t B_{t-1} + A_t A_{t-1} B_{t-2} + ... along dimension 1, by strides of 1, 2, 4, ..."""
    step = 1
    while step < B.shape[1]:
        B = torch.cat([B[:, :step], B[:, step:] + A[:, step:] * B[:, :-step]], 1)
        A = torch.cat([A[:, :step], A[:, step:] * A[:, :-step]], 1)
        step *= 2
    return B


def _plain_scan(s):
    c = s["case"]
    n, d, g = c["n"], c["d"], c["gates"]
    m = d // g
    row, ok = _places(s, c["reverse"])
    x = torch.where(ok[..., None, None], s["x"][row].float().view(n, -1, g, m), 0)
    a = s["a"][row].float()[..., None]
    h0 = None if s["h0"] is None else s["h0"].view(n, g, m)
    if c["dir"] == "forward":
        A = torch.where(ok[..., None, None], a, 1)
        B = x * (1 - A) if c["mix"] else x
        if h0 is not None:
            B[:, 0] += A[:, 0] * h0
        B = _doubling(A, B).view(n, -1, d)
        h = torch.empty_like(s["x"])
        h[row[ok]] = B[ok].to(h.dtype)
        return dict(h=h, h_last=B[:, -1].contiguous())
    back, ok_b = _places(s, not c["reverse"])
    A = torch.cat([torch.ones_like(a[:, :1]), s["a"][back].float()[:, :-1, :, None]], 1)
    B = torch.where(ok_b[..., None, None], s["dh"][back].float().view(n, -1, g, m), 0)
    if s["dh_last"] is not None:
        B[:, 0] += s["dh_last"].view(n, g, m)
    D = torch.zeros((s["x"].shape[0], g, m), device="cuda")
    D[back[ok_b]] = _doubling(A, B)[ok_b]
    D = torch.where(ok[..., None, None], D[row], 0)  # in the recurrence's order
    before = s["h"][row].float().view(n, -1, g, m)[:, :-1]
    before = torch.cat([torch.zeros_like(D[:, :1]) if h0 is None else h0[:, None], before], 1)
    da = (D * (before - x if c["mix"] else before)).sum(3)
    dx = (D * (1 - a) if c["mix"] else D).view(n, -1, d)
    out = dict(da=torch.zeros_like(s["a"]), dx=torch.zeros_like(s["x"]))
    out["da"][row[ok]] = da[ok].to(s["a"].dtype)
    out["dx"][row[ok]] = dx[ok].to(s["x"].dtype)
    if c["state"]:
        out["dh0"] = torch.where(ok[:, :1], (a[:, 0] * D[:, 0]).view(n, d), s["dh_last"])
    return out


def _plain_clip(s):
    total = sum(g.float().square().sum(dtype=torch.float64) for g in s["grads"])
    norm = total.sqrt().float()
    factor = (s["case"]["max_norm"] / norm).clamp_max(1.0)
    out = dict(norm=norm.view(1))
    for t, dt in _DT.items():
        flat = [g.float().mul(factor).to(dt) for g in s["grads"] if g.dtype == dt]
        out[t] = torch.cat(flat) if flat else torch.zeros(0, dtype=dt, device="cuda")
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "gate":
            if c["dir"] == "forward":
                ids, weights = _plain_gate(s["logits"], c["k"], c["renorm"])
                return dict(ids=ids, weights=weights)
            return dict(dlogits=_plain_gate_back(s, c["renorm"]))
        if c["op"] == "layer":
            return dict(out=_plain_layer(s))
        return _plain_scan(s) if c["op"] == "scan" else _plain_clip(s)
    import volume_rendering_amd as v
    if c["op"] == "gate":
        if c["dir"] == "forward":
            ids, weights = s["out"]
            v.nerf_route_gate(s["logits"], ids, weights, renorm=c["renorm"])
            return dict(ids=ids, weights=weights)
        v.nerf_route_gate_grad(s["dweights"], s["logits"], s["ids"], s["weights"], s["dlogits"], renorm=c["renorm"])
        return dict(dlogits=s["dlogits"])
    if c["op"] == "layer":
        v.nerf_routed_mlp(s["x"], s["ids"], s["weights"], s["w1"], s["b1"], s["w2"], s["b2"], s["out"], act=c["act"],
                          workspace=s["ws"])
        return dict(out=s["out"])
    if c["op"] == "scan":
        offsets = s["offsets"] if c["ragged"] else None
        kw = dict(offsets=offsets, n_seq=c["n"], h0=s["h0"], reverse=c["reverse"], mix=c["mix"], workspace=s["ws"])
        if c["dir"] == "forward":
            v.nerf_scan(s["a"], s["x"], s["h"], h_last=s["h_last"], **kw)
            return dict(h=s["h"], h_last=s["h_last"])
        v.nerf_scan_grad(s["dh"], s["a"], s["x"], s["h"], s["da"], s["dx"], dh_last=s["dh_last"], dh0=s["dh0"], **kw)
        out = dict(da=s["da"], dx=s["dx"])
        if c["state"]:
            out["dh0"] = s["dh0"]
        return out
    v.nerf_grad_clip(s["list"], c["max_norm"], s["norm"], workspace=s["ws"])
    return dict(norm=s["norm"], **s["flat"])


def exact(case, seed):
    """The definitions in float64: ranks, pair by pair, step by step."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "gate":
        z = s["logits"].to(f64)
        n, E, k = case["n"], case["experts"], case["k"]
        none = (z == -math.inf).all(1, keepdim=True)
        every = torch.softmax(torch.where(none, 0.0, z), 1).masked_fill(none, 0.0)
        if case["dir"] == "forward":
            left, w = z.clone(), []
            for _ in range(k):  # one choice after the other; argmax takes some largest, whose weight is the same
                best = left.argmax(1, keepdim=True)
                w.append(torch.where(left.gather(1, best) == -math.inf, 0.0, every.gather(1, best)))
                left.scatter_(1, best, -math.inf)
            w = torch.cat(w, 1)
            if case["renorm"]:
                w = w / torch.where(none, 1.0, w.sum(1, keepdim=True))
            return dict(ids=None, weights=w)
        chosen = torch.zeros((n, E), dtype=f64, device="cuda")  # the chosen experts' gradients, by column
        live = s["ids"] >= 0
        for j in range(k):
            col = s["ids"][:, j:j + 1].clamp_min(0).long()
            chosen.scatter_add_(1, col, torch.where(live[:, j:j + 1], s["dweights"][:, j:j + 1].to(f64), 0.0))
        taken = torch.zeros((n, E), dtype=f64, device="cuda")
        taken.scatter_add_(1, s["ids"].clamp_min(0).long(), live.to(f64))
        if case["renorm"]:  # the weights are inputs of the gradient
            w = torch.zeros((n, E), dtype=f64, device="cuda")
            w.scatter_add_(1, s["ids"].clamp_min(0).long(), torch.where(live, s["weights"].to(f64), 0.0))
            return dict(dlogits=w * (chosen - (w * chosen).sum(1, keepdim=True)))
        w = torch.zeros((n, E), dtype=f64, device="cuda")
        w.scatter_add_(1, s["ids"].clamp_min(0).long(), torch.where(live, s["weights"].to(f64), 0.0))
        return dict(dlogits=w * chosen - every * (w * chosen).sum(1, keepdim=True))
    if case["op"] == "layer":
        n, k, hid = case["n"], case["k"], case["hidden"]
        out = torch.zeros((n, case["d_out"]), dtype=f64, device="cuda")
        ids = s["ids"].tolist()
        for t in range(n):
            for j in range(k):
                e = ids[t][j]
                if e < 0:
                    continue
                z = torch.mv(s["w1"][e].to(f64), s["x"][t].to(f64)) + s["b1"][e].to(f64)
                if case["act"] == "gated":
                    z = torch.sigmoid(z[:hid]) * z[:hid] * z[hid:]
                elif case["act"] == "relu":
                    z = torch.relu(z)
                out[t] += s["weights"][t, j].to(f64) * (torch.mv(s["w2"][e].to(f64), z) + s["b2"][e].to(f64))
        return dict(out=out)
    if case["op"] == "scan":
        if s["longest"] > 140000:
            return None
        n, d, g = case["n"], case["d"], case["gates"]
        lo, hi = s["offsets"][:-1].long(), s["offsets"][1:].long()
        x, a = s["x"], s["a"]

        def wide(rows):  # the gates of some rows, one per channel
            return a[rows].to(f64).repeat_interleave(d // g, 1)

        def at(i):  # sequences that have a step i, and its rows
            live = torch.nonzero(hi - lo > i)[:, 0]
            return live, (hi[live] - 1 - i if case["reverse"] else lo[live] + i)

        same = not case["ragged"]
        zero = torch.zeros((n, d), dtype=f64, device="cuda")
        if case["dir"] == "forward":
            state = zero if s["h0"] is None else s["h0"].to(f64)
            h = torch.zeros(x.shape, dtype=f64, device="cuda")
            for i in range(s["longest"]):
                if same:
                    r = hi - 1 - i if case["reverse"] else lo + i
                    old = state
                else:
                    live, r = at(i)
                    old = state[live]
                ar, xr = wide(r), x[r].to(f64)
                new = ar * old + ((1.0 - ar) * xr if case["mix"] else xr)
                h[r] = new
                if same:
                    state = new
                else:
                    state = state.index_copy(0, live, new)
            return dict(h=h, h_last=state)
        flow = zero if s["dh_last"] is None else s["dh_last"].to(f64)  # the gradient at a state from what follows
        da = torch.zeros(a.shape, dtype=f64, device="cuda")
        dx = torch.zeros(x.shape, dtype=f64, device="cuda")
        first = zero if s["h0"] is None else s["h0"].to(f64)
        every = torch.arange(n, device="cuda")
        for i in range(s["longest"] - 1, -1, -1):
            live, r = (every, hi - 1 - i if case["reverse"] else lo + i) if same else at(i)
            before = first[live] if i == 0 else s["h"][r + 1 if case["reverse"] else r - 1].to(f64)
            ar = wide(r)
            D = s["dh"][r].to(f64) + flow[live]
            if case["mix"]:
                before = before - x[r].to(f64)
            da[r] = (D * before).view(-1, g, d // g).sum(2)
            dx[r] = (1.0 - ar) * D if case["mix"] else D
            flow = ar * D if same else flow.index_copy(0, live, ar * D)
        out = dict(da=da, dx=dx)
        if case["state"]:
            out["dh0"] = flow
        return out
    norm = torch.cat([torch.linalg.vector_norm(g.to(f64)).view(1) for g in s["grads"]]).norm().view(1)
    factor = min(1.0, case["max_norm"] / float(norm))
    out = dict(norm=norm)
    for t, dt in _DT.items():
        out[t] = torch.cat([torch.zeros(0, dtype=f64, device="cuda")]
                           + [g.to(f64) * factor for g in s["grads"] if g.dtype == dt])
    return out
