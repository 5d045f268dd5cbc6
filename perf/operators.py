"""The operators of a routed field and its distillation, as measured.

Three operators, each in both directions:

``route``    pairs (sample, choice) sorted by expert, the samples' rows copied
             into that order and the experts' rows summed back with weights
             (forward); the gradients of both (backward).
``expert``   one linear layer per expert on rows sorted by expert (forward);
             its input, weight and bias gradients (backward).
``distill``  Kullback-Leibler loss against a teacher's K largest logits per
             row (``loss``), with the gradient in the same pass (``both``), or
             the gradient from a saved log-sum-exp (``back``).

``run`` computes them in plain torch (float32, rounded once at the end), or
with this repository's entry points where ``own`` is true.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


def listed():
    route = dict(op="route", drop=0.0)
    expert = dict(op="expert", drop=0.0, gather=False, act=False)
    return [
        # one sample through a two-of-sixteen gate: serving, latency only
        dict(route, name="route_token", dir="forward", dtype="bf16", n=1, k=2, experts=16, d=1024),
        # samples of many rays sorted by the cell they lie in, with 63-wide frequency encodings; samples in
        # empty space have no network
        dict(route, name="route_cells", dir="forward", dtype="f32", n=150001, k=1, experts=4096, d=63, drop=0.4),
        # a training batch of 4096 rays x 64 samples, 256 wide, two of eight fields per sample
        dict(route, name="route_field", dir="forward", dtype="bf16", n=262144, k=2, experts=8, d=256),
        dict(route, name="route_field_back", dir="backward", dtype="bf16", n=262144, k=2, experts=8, d=256),
        # gradients at odd sizes: an uneven last batch, rows of no round width, pairs over a capacity dropped
        dict(route, name="route_ragged_back", dir="backward", dtype="f32", n=20011, k=3, experts=61, d=333, drop=0.1),
        # the layer behind route_token: the weights of two experts are read for two rows
        dict(expert, name="expert_token", dir="forward", dtype="bf16", n=1, k=2, experts=16, d_in=1024, d_out=4096,
             gather=True, act=True),
        # a hidden layer of eight 256-wide fields on a training batch
        dict(expert, name="expert_field", dir="forward", dtype="bf16", n=131072, k=2, experts=8, d_in=256, d_out=256,
             act=True),
        # wide experts with uneven loads, rows read through the routing: bound by the matrix units
        dict(expert, name="expert_wide", dir="forward", dtype="bf16", n=16384, k=2, experts=16, d_in=1024, d_out=4096,
             gather=True, act=True),
        dict(expert, name="expert_wide_back", dir="backward", dtype="bf16", n=16384, k=2, experts=16, d_in=1024,
             d_out=4096, gather=True),
        # the first layer of one tiny network per cell (63 -> 32), thousands of short ragged groups
        dict(expert, name="expert_cells_back", dir="backward", dtype="f32", n=150001, k=1, experts=4096, d_in=63,
             d_out=32, drop=0.4),
        # the loss of a single row over many classes: few rows, one long axis
        dict(op="distill", name="distill_row", dir="loss", dtype="f32", n=1, classes=50001, top=16, temperature=1.0),
        # a training batch against a large teacher's top logits: loss and gradient in one pass
        dict(op="distill", name="distill_batch", dir="both", dtype="bf16", n=4096, classes=128000, top=64,
             temperature=2.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 5e12, w["flops"] / (1e15 if c["dtype"] == "bf16" else 1e14))


def draw(rng):
    cap = {}
    for c in listed():
        cap[c["op"]] = max(cap.get(c["op"], 0.0), _cost(c))
    while True:
        op = rng.choice(["route", "expert", "distill"])
        c = dict(op=op, dtype=rng.choice(["f32", "bf16"]))
        if op == "distill":
            c.update(dir=rng.choice(["loss", "both", "back"]), n=_log_int(rng, 1, 16384),
                     classes=_log_int(rng, 32, 262144), top=_log_int(rng, 1, 128),
                     temperature=rng.choice([0.5, 1.0, 2.0, 4.0]))
            c["top"] = min(c["top"], c["classes"])
        else:
            c.update(dir=rng.choice(["forward", "backward"]), k=rng.randint(1, 6), n=_log_int(rng, 1, 262144),
                     drop=rng.choice([0.0, 0.0, 0.1, 0.5]))
            c["experts"] = max(c["k"], _log_int(rng, 1, 4096))
            if op == "route":
                c["d"] = _log_int(rng, 8, 2048)
            else:
                c.update(d_in=_log_int(rng, 16, 2048), d_out=_log_int(rng, 16, 4096),
                         gather=rng.choice([False, True]), act=rng.choice([False, True]))
                if rng.random() < 0.5:  # round widths as often as odd ones
                    c["d_in"], c["d_out"] = (v + 31 & ~31 for v in (c["d_in"], c["d_out"]))
                if c["experts"] * c["d_in"] * c["d_out"] > 1 << 26:
                    continue
        if _cost(c) <= cap[op]:
            return c


def work(case):
    b, n = _SIZE[case["dtype"]], case["n"]
    if case["op"] == "distill":
        full = n * case["classes"] * b
        teacher = n * case["top"] * 8
        both = case["dir"] != "loss"
        return {"bytes": full * (2 if both else 1) + teacher + 8 * n,
                "flops": n * case["classes"] * (6 if both else 4)}
    k, slots = case["k"], n * case["k"]
    live = slots * (1 - case["drop"])
    if case["op"] == "route":
        row = case["d"] * b
        if case["dir"] == "forward":  # ids in; plan out; x in, sorted rows out; expert rows in, sums out
            byt = 12 * slots + 4 * case["experts"] + n * row + slots * row + live * row + 4 * slots + n * row
            return {"bytes": byt, "flops": 2 * live * case["d"]}
        # dout and expert rows in, their gradients out; the sorted rows' gradients in, the samples' out
        byt = 12 * slots + n * row + live * row + slots * row + live * row + n * row
        return {"bytes": byt, "flops": 4 * live * case["d"]}
    din, dout = case["d_in"], case["d_out"]
    touched = min(case["experts"], slots) * din * dout
    xrows = min(n, live) if case["gather"] else live
    if case["dir"] == "forward":
        return {"bytes": xrows * din * b + touched * b + slots * dout * b, "flops": 2 * live * din * dout}
    return {"bytes": live * dout * b + xrows * din * b + touched * b + slots * din * b
            + case["experts"] * (din + 1) * dout * 4, "flops": 4 * live * din * dout}


def _expert_ids(case, gen):
    """[n, k] int32: distinct experts per sample, uneven loads, -1 for a pair without an expert."""
    n, k, E = case["n"], case["k"], case["experts"]
    u = torch.rand(E, generator=gen, device="cuda")
    if E <= 64:  # a gate's loads fall off by rank
        p = (torch.argsort(u).float() + 1.0) ** -0.7
    else:        # cells of a scene: about a third hold no sample
        p = (u - 0.3).clamp_min(0.0) + 1e-6
    first = torch.multinomial(p, n, replacement=True, generator=gen)
    if k > 1:
        step = torch.randint(1, (E - 1) // (k - 1) + 1, (n, k - 1), generator=gen, device="cuda")
        ids = (first[:, None] + torch.cat([torch.zeros_like(step[:, :1]), step.cumsum(1)], 1)) % E
    else:
        ids = first[:, None]
    if case["drop"]:
        ids = torch.where(torch.rand(n, k, generator=gen, device="cuda") < case["drop"], -1, ids)
    return ids.to(torch.int32).contiguous()


def _plan(ids, E):
    flat = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    key, order = torch.sort(flat, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.searchsorted(key, torch.arange(E + 1, dtype=key.dtype, device=key.device))
    return offsets.to(torch.int32), order.to(torch.int32), place.to(torch.int32).view(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DT[case["dtype"]]
    n = case["n"]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    def empty(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = dict(case=case)
    if case["op"] == "distill":
        V, K = case["classes"], case["top"]
        s["logits"] = torch.empty((n, V), dtype=dt, device="cuda")
        for a in range(0, n, 512):
            s["logits"][a:a + 512] = normal(min(512, n - a), V, scale=2.0)
        s["t_logits"] = normal(n, K, scale=2.0, dtype=torch.float32).sort(dim=1, descending=True).values.add_(6.0)
        ids = torch.randint(0, V, (n, 1), generator=gen, device="cuda") + torch.arange(K, device="cuda") * max(1, V // K)
        ids = ids % V
        pad = torch.rand(n, K, generator=gen, device="cuda") < 0.02
        if n > 1:  # rows outside the loss have no teacher entries
            pad |= torch.rand(n, 1, generator=gen, device="cuda") < 0.03
        s["t_ids"] = torch.where(pad, -1, ids).to(torch.int32).contiguous()
        s["row_scale"] = torch.rand(n, generator=gen, device="cuda").add_(0.5).mul_(1.0 / n)
        if case["dir"] == "back":
            s["lse"] = torch.cat([torch.logsumexp(s["logits"][a:a + 512].float() / case["temperature"], 1)
                                  for a in range(0, n, 512)])
        if own:
            s["loss"], s["lse_out"] = empty(n, dtype=torch.float32), empty(n, dtype=torch.float32)
            s["grad"] = empty(n, V) if case["dir"] != "loss" else None
            import volume_rendering_amd as v
            s["ws"] = empty(max(1, v.nerf_distill_workspace_size(n, V)), dtype=torch.uint8)
        return s
    k, E = case["k"], case["experts"]
    S = n * k
    ids = _expert_ids(case, gen)
    plan = _plan(ids, E)
    if case["op"] == "route":
        d = case["d"]
        s["ids"] = ids
        s["weights"] = torch.rand(n, k, generator=gen, device="cuda").add_(0.05)
        s["weights"] /= s["weights"].sum(1, keepdim=True)
        s["y"] = normal(S, d)
        if case["dir"] == "forward":
            s["x"] = normal(n, d)
        else:
            s["offsets"], s["order"], s["place"] = plan
            s["dout"], s["drows"] = normal(n, d), normal(S, d)
        if own:
            import volume_rendering_amd as v
            i32 = torch.int32
            if case["dir"] == "forward":
                s["plan"] = (empty(E + 1, dtype=i32), empty(S, dtype=i32), empty(n, k, dtype=i32))
                s["rows"], s["out"] = empty(S, d), empty(n, d)
                s["ws"] = empty(max(1, v.nerf_route_workspace_size(n, k, E)), dtype=torch.uint8)
            else:
                s["dy"], s["dw"], s["dx"] = empty(S, d), empty(n, k, dtype=torch.float32), empty(n, d)
        return s
    din, dout = case["d_in"], case["d_out"]
    s["offsets"], s["order"] = plan[:2]
    s["bounds"] = s["offsets"].tolist()
    s["x"] = normal(n if case["gather"] else S, din).relu_()
    s["weight"] = normal(E, dout, din, scale=math.sqrt(2.0 / din))
    if case["dir"] == "forward":
        s["bias"] = normal(E, dout, scale=0.1, dtype=torch.float32)
    else:
        s["dz"] = normal(S, dout)
    if own:
        import volume_rendering_amd as v
        if case["dir"] == "forward":
            s["out"] = empty(S, dout)
        else:
            s["dx"] = empty(S, din)
            s["dweight"], s["dbias"] = empty(E, dout, din, dtype=torch.float32), empty(E, dout, dtype=torch.float32)
            s["ws"] = empty(max(1, v.nerf_expert_linear_grad_workspace_size(S, E, din, dout)), dtype=torch.uint8)
    return s


def _plain_route(s):
    c = s["case"]
    k, E, dt = c["k"], c["experts"], s["y"].dtype
    if c["dir"] == "forward":
        offsets, order, place = _plan(s["ids"], E)
        live_slot = torch.arange(order.numel(), device="cuda") < offsets[E]
        rows = torch.where(live_slot[:, None], s["x"][(order // k).long()], 0)
        live = place < offsets[E]
        out = 0
        for j in range(k):
            row = s["y"][place[:, j].long()].float() * s["weights"][:, j:j + 1]
            out = out + torch.where(live[:, j:j + 1], row, 0)
        return dict(offsets=offsets, order=order, place=place, rows=rows, out=out.to(dt))
    place, order, offsets = s["place"], s["order"], s["offsets"]
    live_slot = (torch.arange(order.numel(), device="cuda") < offsets[E])[:, None]
    g = s["dout"][(order // k).long()].float()
    w = s["weights"].reshape(-1)[order.long()][:, None]
    dy = torch.where(live_slot, g * w, 0).to(dt)
    dw_slot = torch.where(live_slot[:, 0], (g * s["y"].float()).sum(1), 0)
    dw = dw_slot[place.long()]
    drows = torch.where(live_slot, s["drows"].float(), 0)
    dx = 0
    for j in range(k):
        dx = dx + drows[place[:, j].long()]
    return dict(dy=dy, dweights=dw, dx=dx.to(dt))


def _plain_expert(s):
    c = s["case"]
    E, b, dt = c["experts"], s["bounds"], s["x"].dtype
    S = c["n"] * c["k"]
    x = s["x"].float()
    if c["gather"]:
        x = x[(s["order"] // c["k"]).long()]
    W = s["weight"].float()
    forward = c["dir"] == "forward"
    dz = None if forward else s["dz"].float()
    if forward:
        y = torch.zeros((S, c["d_out"]), dtype=torch.float32, device="cuda")
    else:
        dx = torch.zeros((S, c["d_in"]), dtype=torch.float32, device="cuda")
        dW, db = torch.zeros_like(W), torch.zeros(W.shape[:2], dtype=torch.float32, device="cuda")
    if E <= 64:  # few experts: one product each
        for e in range(E):
            r = slice(b[e], b[e + 1])
            if b[e] == b[e + 1]:
                continue
            if forward:
                y[r] = x[r] @ W[e].t() + s["bias"][e]
            else:
                dx[r] = dz[r] @ W[e]
                dW[e] = dz[r].t() @ x[r]
                db[e] = dz[r].sum(0)
    else:        # many: short groups padded to the longest, batched
        longest = max(1, max(b[e + 1] - b[e] for e in range(E)))
        off = s["offsets"].long()
        step = max(1, (1 << 28) // (longest * max(c["d_in"], c["d_out"]) + c["d_in"] * c["d_out"]))
        for a in range(0, E, step):
            lo, hi = off[a:min(E, a + step)], off[a + 1:min(E, a + step) + 1]
            idx = lo[:, None] + torch.arange(longest, device="cuda")
            ok = idx < hi[:, None]
            idx = idx.clamp_max(S - 1)
            xe = torch.where(ok[..., None], x[idx], 0)
            We = W[a:a + step]
            if forward:
                ye = torch.bmm(xe, We.transpose(1, 2).contiguous()) + s["bias"][a:a + step, None]
                y[idx[ok]] = ye[ok]
            else:
                ze = torch.where(ok[..., None], dz[idx], 0)
                dx[idx[ok]] = torch.bmm(ze, We)[ok]
                dW[a:a + step] = torch.bmm(ze.transpose(1, 2).contiguous(), xe)
                db[a:a + step] = ze.sum(1)
    if forward:
        return dict(y=(y.relu_() if c["act"] else y).to(dt))
    if c["act"]:
        dx = torch.where(x > 0, dx, 0)
    return dict(dx=dx.to(dt), dweight=dW, dbias=db)


def _plain_distill(s):
    c = s["case"]
    T, V = c["temperature"], c["classes"]
    z = s["logits"].float() / T
    if c["dir"] == "back":
        lse = s["lse"]
    else:
        m = z.amax(1, keepdim=True)
        lse = (m + (z - m).exp().sum(1, keepdim=True).log())[:, 0]
    has = s["t_ids"] >= 0
    idx = s["t_ids"].clamp_min(0).long()
    t = torch.where(has, s["t_logits"] / T, -math.inf)
    tm = t.amax(1, keepdim=True).clamp_min(-3e38)
    e = (t - tm).exp()
    tot = e.sum(1, keepdim=True)
    p = torch.where(tot > 0, e / tot, 0)
    out = {}
    if c["dir"] != "back":
        logp = t - tm - torch.where(tot > 0, tot, 1).log()
        logq = z.gather(1, idx) - lse[:, None]
        out["loss"] = T * T * torch.where(p > 0, p * (logp - logq), 0).sum(1)
        out["lse"] = lse
    if c["dir"] != "loss":
        g = (z - lse[:, None]).exp_().mul_(p.sum(1, keepdim=True))
        g.scatter_add_(1, idx, -p)
        out["grad"] = g.mul_(T * s["row_scale"][:, None]).to(s["logits"].dtype)
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"route": _plain_route, "expert": _plain_expert, "distill": _plain_distill}[c["op"]](s)
    import volume_rendering_amd as v
    if c["op"] == "route":
        if c["dir"] == "forward":
            offsets, order, place = s["plan"]
            v.nerf_route_plan(s["ids"], c["experts"], offsets, order, place, workspace=s["ws"])
            v.nerf_route_gather(s["x"], offsets, place, s["rows"])
            v.nerf_route_combine(s["y"], offsets, place, s["weights"], s["out"])
            return dict(offsets=offsets, order=order, place=place, rows=s["rows"], out=s["out"])
        v.nerf_route_combine_grad(s["dout"], s["y"], s["offsets"], s["place"], s["weights"], s["dy"], s["dw"])
        v.nerf_route_combine(s["drows"], s["offsets"], s["place"], None, s["dx"])
        return dict(dy=s["dy"], dweights=s["dw"], dx=s["dx"])
    if c["op"] == "expert":
        order, k = (s["order"], c["k"]) if c["gather"] else (None, 1)
        if c["dir"] == "forward":
            v.nerf_expert_linear(s["x"], s["weight"], s["bias"], s["offsets"], s["out"], order=order, k=k,
                                 relu=c["act"])
            return dict(y=s["out"])
        v.nerf_expert_linear_grad(s["dz"], s["x"], s["weight"], s["offsets"], s["dx"], s["dweight"], s["dbias"],
                                  order=order, k=k, relu_x=c["act"], workspace=s["ws"])
        return dict(dx=s["dx"], dweight=s["dweight"], dbias=s["dbias"])
    if c["dir"] == "back":
        v.nerf_distill_topk_grad(s["logits"], s["t_logits"], s["t_ids"], c["temperature"], s["lse"], s["grad"],
                                 row_scale=s["row_scale"])
        return dict(grad=s["grad"])
    v.nerf_distill_topk(s["logits"], s["t_logits"], s["t_ids"], c["temperature"], s["loss"], lse=s["lse_out"],
                        grad=s["grad"], row_scale=s["row_scale"], workspace=s["ws"])
    out = dict(loss=s["loss"], lse=s["lse_out"])
    if c["dir"] == "both":
        out["grad"] = s["grad"]
    return out


def exact(case, seed):
    """The definitions in float64, pair by pair of index sets rather than through the sorted order."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "distill":
        T, n = case["temperature"], case["n"]
        res = dict(loss=[], lse=[], grad=[])
        for a in range(0, n, 256):
            z = s["logits"][a:a + 256].to(f64) / T
            idx = s["t_ids"][a:a + 256].long()
            t = s["t_logits"][a:a + 256].to(f64) / T
            t[idx < 0] = -math.inf
            none = (idx < 0).all(1)
            t[none] = 0.0
            logp = torch.log_softmax(t, 1)
            p = logp.exp()
            p[none] = 0.0
            p[idx < 0] = 0.0
            lse = torch.logsumexp(z, 1) if case["dir"] != "back" else s["lse"][a:a + 256].to(f64)
            dense = torch.zeros_like(z).scatter_add_(1, idx.clamp_min(0), p)
            logq = z - lse[:, None]
            # sum of p ln p - p ln q; entries of no mass add nothing
            res["loss"].append(T * T * (torch.where(p > 0, p * logp, 0.0).sum(1) - (dense * logq).sum(1)))
            res["lse"].append(lse)
            if case["dir"] != "loss":
                scale = s["row_scale"][a:a + 256].to(f64)[:, None] * T
                res["grad"].append(scale * (logq.exp() * p.sum(1, keepdim=True) - dense))
        keep = {"loss": ["loss", "lse"], "both": ["loss", "lse", "grad"], "back": ["grad"]}[case["dir"]]
        return {key: torch.cat(res[key]) for key in keep}
    k, E, n = case["k"], case["experts"], case["n"]
    S = n * k
    if case["op"] == "route":
        fwd = case["dir"] == "forward"
        if fwd:  # a pair's slot is its rank by (expert, pair); pairs without an expert come last
            key = s["ids"].cpu().to(torch.int64).reshape(-1)
            key = torch.where(key < 0, E, key) * S + torch.arange(S)
            place = torch.empty(S, dtype=torch.int64).scatter_(0, key.argsort(), torch.arange(S)).cuda()
            last = int((s["ids"] >= 0).sum())
        else:
            place, last = s["place"].long().reshape(-1), int(s["offsets"][E])
        pair = torch.nonzero(place < last)[:, 0]
        slot, tok = place[pair], pair // k
        w = s["weights"].to(f64).reshape(-1)
        d = case["d"]
        if fwd:
            rows = torch.zeros((S, d), dtype=f64, device="cuda")
            rows[slot] = s["x"].to(f64)[tok]
            out = torch.zeros((n, d), dtype=f64, device="cuda")
            out.index_add_(0, tok, s["y"].to(f64)[slot] * w[pair][:, None])
            return dict(offsets=None, order=None, place=None, rows=rows, out=out)
        g = s["dout"].to(f64)[tok]
        dy = torch.zeros((S, d), dtype=f64, device="cuda")
        dy[slot] = g * w[pair][:, None]
        dw = torch.zeros(S, dtype=f64, device="cuda")
        dw[pair] = (g * s["y"].to(f64)[slot]).sum(1)
        dx = torch.zeros((n, d), dtype=f64, device="cuda")
        dx.index_add_(0, tok, s["drows"].to(f64)[slot])
        return dict(dy=dy, dweights=dw.view(n, k), dx=dx)
    b, fwd = s["bounds"], case["dir"] == "forward"
    tok = (s["order"] // k).long() if case["gather"] else torch.arange(S, device="cuda")
    W = s["weight"]
    if fwd:
        y = torch.zeros((S, case["d_out"]), dtype=f64, device="cuda")
    else:
        dx = torch.zeros((S, case["d_in"]), dtype=f64, device="cuda")
        dW = torch.zeros(W.shape, dtype=f64, device="cuda")
        db = torch.zeros(W.shape[:2], dtype=f64, device="cuda")
    for e in range(E):
        lo, hi = b[e], b[e + 1]
        if lo == hi:
            continue
        xe, We = s["x"][tok[lo:hi]].to(f64), W[e].to(f64)
        if fwd:
            ye = torch.mm(xe, We.t()).add_(s["bias"][e].to(f64))
            y[lo:hi] = ye.clamp_min_(0.0) if case["act"] else ye
        else:
            ze = s["dz"][lo:hi].to(f64)
            dxe = torch.mm(ze, We)
            dx[lo:hi] = dxe * (xe > 0) if case["act"] else dxe
            dW[e] = torch.mm(ze.t(), xe)
            db[e] = ze.sum(0)
    return dict(y=y) if fwd else dict(dx=dx, dweight=dW, dbias=db)
