"""The gated linear recurrence and its gradient on the GPU against the float64
oracle (oracle/streaming.py).

Bounds.  Every state is a sum of terms that are products of gates and one input;
M_t = |a_t| M_{t-1} + |b_t| is the sum of their magnitudes.  A term takes one
rounding per step, and joins of runs of eight steps at most 14 more per run (six
between lanes, eight between waves), so fewer than four a step; (1 - a) x takes
two.  With half a step of float32 being 2^-24,
  E_t = |a_t| E_{t-1} + 8 2^-24 M_t
covers them with a factor of about two.  A bfloat16 result is off by another 2^-8
of itself.  Gate gradients are sums of m products of a state's gradient (error E)
and h - x (exact inputs): sum E |h - x| + (m + 4) 2^-24 sum |D| |h - x|.
"""
import numpy as np
import pytest

from oracle import streaming as O
from tests.gpu_util import host, say, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _f64(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def _dt(name):
    torch = torch_cuda()
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _put(a, dtype, pad=0):
    """Device tensor of a numpy array; with `pad`, rows further apart that start at an odd element."""
    torch = torch_cuda()
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(_dt(dtype))
    if not pad:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    big[:, 1:1 + t.shape[1]] = t
    return big[:, 1:1 + t.shape[1]]


def _offsets(g, lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def _inputs(g, rows, d, gates, n):
    a = 1.0 / (1.0 + np.exp(-(2.0 + 1.5 * g.standard_normal((rows, gates)))))
    a[g.random(a.shape) < 0.02] = 0.0  # (a state that is dropped)
    a[g.random(a.shape) < 0.02] = 1.0
    a *= np.where(g.random(a.shape) < 0.1, -1.0, 1.0)
    return a, g.standard_normal((rows, d)), g.standard_normal((n, d))


def _bounds(a, b, offsets, start, reverse):
    """M and E per row, and E of the last states."""
    d = b.shape[1]
    A = np.abs(np.repeat(a, d // a.shape[1], axis=1))
    M, E, last = np.zeros(b.shape), np.zeros(b.shape), np.zeros(start.shape)
    for s in range(len(offsets) - 1):
        m, e = np.abs(start[s]), np.zeros(d)
        for r in O._rows(offsets[s], offsets[s + 1], reverse):
            m = A[r] * m + np.abs(b[r])
            e = A[r] * e + 8 * U * m
            M[r], E[r] = m, e
        last[s] = e
    return M, E, last


def _close(what, got, ref, tol):
    live = ~np.isnan(ref)
    worst = np.max(np.abs(got - ref)[live] / (tol[live] + 1e-30)) if live.any() else 0.0
    say(f"  {what}: {worst:.2f} of the bound")
    assert (np.abs(got - ref)[live] <= tol[live] + 1e-30).all(), what


TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]
# lengths, d, gates, reverse, mix
CASES = [
    ([1], 1, 1, False, False),
    ([1, 1, 1, 1, 1], 40, 40, False, True),
    ([0, 3, 0, 8, 9, 1, 0], 3, 3, True, False),
    ([63, 64, 65, 7, 0, 200], 2, 2, False, True),
    ([5, 130, 64, 0, 17], 16, 1, True, True),
    ([70, 3, 129], 33, 33, True, False),
    ([70, 3, 129], 33, 11, False, True),       # three channels a gate: fewer than a piece
    ([40, 0, 300], 63, 9, True, True),          # seven
    ([64, 511, 33], 257, 257, False, False),    # one channel past a block
    ([30, 64], 256, 4, False, True),
    ([25, 1, 90], 600, 1, True, True),          # a gate over several blocks
    ([33, 20], 1030, 2, False, False),
    ([18] * 50, 96, 96, False, True),
    ([2 + i % 40 for i in range(300)], 24, 3, True, True),
    ([4100], 5, 5, False, True),                # long: split into chunks
    ([6000, 0, 1, 3000], 70, 70, True, False),
    ([5000, 37], 130, 1, True, True),
    ([9001], 600, 2, False, True),
    ([3, 0, 4, 2, 1, 4, 4, 3], 600, 1, True, True),      # walked alone, a gate over several blocks
    ([1, 2, 0, 3, 4, 4, 4, 5], 24, 3, False, True),      # alone, gates side by side
    ([4, 1, 0, 2], 1030, 1030, True, False),
    ([120, 200, 0, 65, 64, 130], 256, 2, False, True),   # several tiles of eight waves
    ([120, 200, 0, 65, 64, 128], 256, 256, True, True),
]


def _equal(lens):
    return len(set(lens)) == 1


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_scan_and_gradient(case, dtype, gate_dtype, pad):
    _check(case, CASES[case], dtype, gate_dtype, pad)


def _ragged(n, top, seed):
    return [int(v) for v in np.random.default_rng(seed).integers(0, top + 1, n)]


# lengths, d, gates, reverse, mix, type, gates' type, pad
LARGE = [
    (_ragged(700, 24, 1), 256, 256, False, True, "bf16", "bf16", 0),   # many short ones: a lane's channels each
    (_ragged(700, 24, 2), 256, 8, True, True, "f32", "f32", 3),
    (_ragged(9000, 16, 3), 13, 1, False, False, "bf16", "f32", 0),
    (_ragged(17000, 12, 4), 2, 2, True, True, "f32", "f32", 0),
    ([40] * 8200, 4, 2, False, True, "bf16", "bf16", 1),               # rows of a few bytes
    (_ragged(16, 280, 5), 1024, 1024, False, True, "bf16", "bf16", 0),  # fewer channels a workgroup
    (_ragged(16, 280, 6), 1024, 16, True, False, "f32", "f32", 3),
    (_ragged(20, 330, 7), 1026, 9, True, True, "bf16", "f32", 0),
    (_ragged(70, 1400, 8), 64, 64, True, True, "bf16", "bf16", 0),      # chunks of more sequences than lanes
    (_ragged(70, 330, 9), 256, 1, False, True, "f32", "f32", 0),
    (_ragged(130, 200, 10), 160, 1, False, True, "f32", "f32", 0),      # whole ones of a gate of 40 lanes
    ([9100], 256, 1, True, True, "bf16", "f32", 0),                    # more chunks than are looked at together
    ([3000] * 4, 64, 64, False, True, "f32", "f32", 0),                # chunks of several sequences side by side
    ([0, 9000, 0, 0, 1], 24, 24, False, True, "bf16", "bf16", 3),
]


@pytest.mark.parametrize("case", range(len(LARGE)))
def test_scan_and_gradient_of_many_sequences(case):
    *shape, dtype, gate_dtype, pad = LARGE[case]
    _check(100 + case, shape, dtype, gate_dtype, pad)


def _check(case, shape, dtype, gate_dtype, pad):
    torch = torch_cuda()
    import volume_rendering_amd as v
    lens, d, gates, reverse, mix = shape
    say(f"scan case={case} {dtype}/{gate_dtype} pad={pad} rows={sum(lens)} d={d} gates={gates}")
    g = np.random.default_rng([case, 1])
    behind = 5 if pad else 0  # rows behind the last sequence, left as they are
    off = _offsets(g, lens)
    rows, n = int(off[-1]) + behind, len(lens)
    a, x, h0 = _inputs(g, rows, d, gates, n)
    ta, tx, th0 = _put(a, gate_dtype, pad), _put(x, dtype, pad), _put(h0, "f32")
    a, x = _f64(ta), _f64(tx)
    use_state = case % 3 != 1
    ho = _f64(th0) if use_state else None
    toff = torch.from_numpy(off.astype(np.int32)).cuda() if (not _equal(lens) or behind) else None
    kw = dict(offsets=toff, n_seq=n, h0=th0 if use_state else None, reverse=reverse, mix=mix)

    big = torch.full((rows, d + pad), 7.0, dtype=_dt(dtype), device="cuda")
    h = big[:, 1:1 + d] if pad else big
    last = torch.full((n, d), 7.0, device="cuda")
    v.nerf_scan(ta, tx, h, h_last=last, **kw)
    ref, ref_last = O.scan(a, x, off, ho, reverse, mix)
    A = np.repeat(a, d // gates, axis=1)
    b = (1.0 - A) * x if mix else x
    _, E, E_last = _bounds(a, b, off, np.zeros((n, d)) if ho is None else ho, reverse)
    hh = _f64(h)
    _close("h", hh, ref, E + HALF[dtype] * (np.abs(ref) + E))
    _close("h_last", _f64(last), ref_last, E_last + U * np.abs(ref_last))
    if behind:
        assert (hh[int(off[-1]):] == 7.0).all() and (_f64(big)[:, 0] == 7.0).all()

    # the gradient, of the states as they were returned
    dh, dl = g.standard_normal((rows, d)), g.standard_normal((n, d))
    tdh, tdl = _put(dh, dtype, pad), _put(dl, "f32")
    dh, dl = _f64(tdh), _f64(tdl) if use_state else None
    da = torch.full((rows, gates), 7.0, dtype=_dt(gate_dtype), device="cuda")
    dx = torch.full((rows, d), 7.0, dtype=_dt(dtype), device="cuda")
    dh0 = torch.full((n, d), 7.0, device="cuda")
    v.nerf_scan_grad(tdh, ta, tx if mix else None, h, da, dx, dh_last=tdl if use_state else None, dh0=dh0, **kw)
    hz = np.nan_to_num(hh)
    rda, rdx, rdh0 = O.scan_grad(dh, dl, a, x, hz, ho, off, reverse, mix)
    # D_t = dh_t + a_{t+1} D_{t+1}: the recurrence with a_t dh_t on what flows in, against the sequence
    start = np.zeros((n, d)) if dl is None else dl
    flow_m, flow_e, E0 = _bounds(a, A * dh, off, start, not reverse)
    before_m, before_e = np.zeros((rows, d)), np.zeros((rows, d))  # of what flows into each row
    prev = np.zeros((rows, d))
    for s in range(n):
        order = list(O._rows(off[s], off[s + 1], reverse))
        for i, r in enumerate(order):
            nxt = order[i + 1] if i + 1 < len(order) else None
            before_m[r] = np.abs(start[s]) if nxt is None else flow_m[nxt]
            before_e[r] = 0.0 if nxt is None else flow_e[nxt]
            prev[r] = (0.0 if ho is None else ho[s]) if i == 0 else hz[order[i - 1]]
    D_m, D_e = np.abs(dh) + before_m, before_e + U * (np.abs(dh) + before_m)
    factor = np.abs(1.0 - A) if mix else np.ones_like(A)
    e = factor * (D_e + 2 * U * D_m)
    _close("dx", _f64(dx), rdx, e + HALF[dtype] * (np.abs(np.nan_to_num(rdx)) + e))
    # (h - x is rounded once)
    diff = np.abs(prev - x) if mix else np.abs(prev)
    m = d // gates
    e = ((D_e + (m + 5) * U * D_m) * diff).reshape(rows, gates, m).sum(2)
    _close("da", _f64(da), rda, e + HALF[gate_dtype] * (np.abs(np.nan_to_num(rda)) + e))
    _close("dh0", _f64(dh0), rdh0, E0 + 2 * U * (np.abs(rdh0) + E0))
    if behind:
        assert (_f64(da)[int(off[-1]):] == 7.0).all() and (_f64(dx)[int(off[-1]):] == 7.0).all()


def test_empty_calls_and_sequences():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("scan of nothing")
    z = torch.empty((0, 6), device="cuda")
    h0, last, off = torch.randn((3, 6), device="cuda"), torch.zeros((3, 6), device="cuda"), torch.zeros(
        4, dtype=torch.int32, device="cuda")
    v.nerf_scan(z, z, torch.empty_like(z), h0=h0, h_last=last, offsets=off)
    assert torch.equal(last, h0)
    last.zero_()
    v.nerf_scan(z, z, torch.empty_like(z), h0=h0, h_last=last, n_seq=3)
    assert torch.equal(last, h0)
    dl, d0 = torch.randn((3, 6), device="cuda"), torch.zeros((3, 6), device="cuda")
    v.nerf_scan_grad(z, z, None, torch.empty_like(z), torch.empty_like(z), torch.empty_like(z), dh_last=dl, dh0=d0,
                     offsets=off)
    assert torch.equal(d0, dl)
    v.nerf_scan(z, z, torch.empty_like(z), offsets=off[:1])  # no sequences
    wide, gate = torch.empty((0, 600), device="cuda"), torch.empty((0, 1), device="cuda")  # a gate over several blocks
    dl, d0 = torch.randn((3, 600), device="cuda"), torch.zeros((3, 600), device="cuda")
    v.nerf_scan_grad(wide, gate, None, torch.empty_like(wide), torch.empty_like(gate), torch.empty_like(wide),
                     dh_last=dl, dh0=d0, offsets=off)
    assert torch.equal(d0, dl)


@pytest.mark.parametrize("d", [8, 257, 1024])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_stream_step_in_place_equals_the_sequence(dtype, d):
    """Length-1 calls that update a state in place reproduce one long call."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"scan step {dtype} d={d}")
    g = np.random.default_rng(d)
    n, steps = 37, 12
    a, x, h0 = _inputs(g, n * steps, d, d, n)
    ta, tx = _put(a, "f32").view(n, steps, d), _put(x, dtype).view(n, steps, d)
    state = _put(h0, "f32")
    whole, last = torch.empty((n * steps, d), dtype=_dt(dtype), device="cuda"), torch.empty((n, d), device="cuda")
    v.nerf_scan(ta.view(-1, d), tx.view(-1, d), whole, h0=state, h_last=last, n_seq=n, mix=True)
    out = torch.empty((n, d), dtype=_dt(dtype), device="cuda")
    M = np.abs(_f64(state))
    for i in range(steps):
        v.nerf_scan(ta[:, i], tx[:, i], out, h0=state, h_last=state, n_seq=n, mix=True)  # (rows steps * d apart)
        ai, xi = _f64(ta[:, i]), _f64(tx[:, i])
        M = np.abs(ai) * M + np.abs((1 - ai) * xi)
        tol = 16 * (i + 1) * U * M
        ref = _f64(whole.view(n, steps, d)[:, i])
        assert (np.abs(_f64(out) - ref) <= tol + 2 * HALF[dtype] * (np.abs(ref) + tol)).all()
    assert (np.abs(_f64(state) - _f64(last)) <= 16 * steps * U * M).all()


@pytest.mark.parametrize("lens", [[9, 0, 20, 33], [3000, 2500]])
def test_not_a_number_stays_in_its_sequence(lens):
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"scan NaN {lens}")
    g = np.random.default_rng(5)
    off = _offsets(g, lens)
    d = 12
    a, x, _ = _inputs(g, int(off[-1]), d, d, len(lens))
    x[off[-2] - 1] = np.nan  # the last row before the last sequence
    x[off[-2]:off[-1]] += 0.0
    ta, tx = _put(a, "f32"), _put(x, "f32")
    h, last = torch.empty_like(tx), torch.empty((len(lens), d), device="cuda")
    v.nerf_scan(ta, tx, h, h_last=last, offsets=torch.from_numpy(off.astype(np.int32)).cuda())
    hh = _f64(h)
    assert np.isnan(hh[off[-2] - 1]).all() and np.isnan(_f64(last)[-2]).all()
    assert np.isfinite(hh[off[-2]:]).all() and np.isfinite(hh[:off[-2] - 1]).all()
    da, dx = torch.empty_like(ta), torch.empty_like(tx)
    v.nerf_scan_grad(tx, ta, None, tx, da, dx, offsets=torch.from_numpy(off.astype(np.int32)).cuda())
    assert np.isfinite(_f64(dx)[off[-2]:]).all() and np.isfinite(_f64(da)[off[-2]:]).all()


def test_infinite_inputs_before_a_closed_gate_and_magnitudes():
    """Values near the type's ends: sums that stay in range are exact to the bound, gates of 0 drop large states."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("scan of large values")
    d, n = 4, 40
    a, x = np.full((n, d), 0.5), np.full((n, d), 1e38)
    a[20] = 0.0
    ta, tx = _put(a, "f32"), _put(x, "f32")
    h = torch.empty_like(tx)
    v.nerf_scan(ta, tx, h)
    ref, _ = O.scan(_f64(ta), _f64(tx), [0, n])
    assert (np.abs(_f64(h) - ref) <= 2.0 ** -20 * ref).all()


def test_offsets_out_of_range_are_kept_in_range():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("scan offsets")
    d = 6
    ta, tx = torch.rand((40, d), device="cuda"), torch.randn((40, d), device="cuda")
    h = torch.full((40, d), 7.0, device="cuda")
    off = torch.tensor([-5, 10, 4, 30, 10 ** 9], dtype=torch.int32, device="cuda")
    v.nerf_scan(ta, tx, h, offsets=off)
    ref, _ = O.scan(_f64(ta), _f64(tx), [0, 10])
    assert np.allclose(_f64(h)[:4], ref[:4], atol=1e-5)
    ref, _ = O.scan(_f64(ta)[30:], _f64(tx)[30:], [0, 10])
    assert np.allclose(_f64(h)[30:], ref, atol=1e-5)


@pytest.mark.parametrize("rows,n,d,gates", [(8192, 1, 64, 64), (3000, 4, 40, 1), (600, 200, 24, 24), (9000, 2, 600, 1)])
def test_repeats_streams_and_workspaces(rows, n, d, gates):
    """Bit-equal results from call to call, on another stream, with the smallest workspace, and replayed."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"scan repeats rows={rows} n={n} d={d} gates={gates}")
    gen = torch.Generator(device="cuda").manual_seed(rows)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda")
    a, x, dh = torch.sigmoid(mk(rows, gates) + 3), mk(rows, d), mk(rows, d)
    h0 = mk(n, d)
    size = v.nerf_scan_workspace_size(rows, d, gates=gates, n_seq=n), v.nerf_scan_workspace_size(
        rows, d, gates=gates, n_seq=n, backward=True)

    def call(ws):
        out = [torch.empty_like(x), torch.empty_like(h0), torch.empty_like(a), torch.empty_like(x), torch.empty_like(h0)]
        v.nerf_scan(a, x, out[0], h0=h0, h_last=out[1], n_seq=n, mix=True, workspace=ws and ws[0])
        v.nerf_scan_grad(dh, a, x, out[0], out[2], out[3], h0=h0, dh_last=h0, dh0=out[4], n_seq=n, mix=True,
                         workspace=ws and ws[1])
        return out

    want = call(None)
    guard = [torch.full((s + 64,), 171, dtype=torch.uint8, device="cuda") for s in size]
    exact = [t[:s] for t, s in zip(guard, size)]
    assert all(torch.equal(p, q) for p, q in zip(call(exact), want))
    torch.cuda.synchronize()
    assert all((t[s:] == 171).all() for t, s in zip(guard, size))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = call(exact)
    stream.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(exact)
    for i in range(3):
        x.mul_(1.25)
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, call(None)))


@pytest.mark.parametrize("d,gates", [(2, 2), (6, 1)])
def test_rows_far_apart(d, gates):
    """Rows so far apart that a wave's tile would leave 32-bit byte offsets."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    rows, ld = 21, (1 << 23) + 5
    say(f"scan of rows {ld} apart, d={d} gates={gates}")
    g = np.random.default_rng(d)
    a, x, _ = _inputs(g, rows, d, gates, 1)
    dh = g.standard_normal((rows, d))
    def far(t, width):
        big = torch.full(((rows - 1) * ld + width,), float("nan"), device="cuda").as_strided((rows, width), (ld, 1))
        return big.copy_(torch.from_numpy(t.astype(np.float32)).cuda()) if t is not None else big
    ta, tx, tdh = far(a, gates), far(x, d), far(dh, d)
    th = far(np.zeros((rows, d)), d)
    off = torch.tensor([0, 3, rows], dtype=torch.int32, device="cuda")
    want = [torch.empty((rows, c), device="cuda") for c in (d, gates, d)]
    near = [t.contiguous() for t in (ta, tx, tdh)]
    for reverse in (False, True):
        v.nerf_scan(ta, tx, th, offsets=off, reverse=reverse, mix=True)
        v.nerf_scan(near[0], near[1], want[0], offsets=off, reverse=reverse, mix=True)
        A, X = _f64(near[0]), _f64(near[1])
        ref, _ = O.scan(A, X, [0, 3, rows], None, reverse, True)
        _, E, _ = _bounds(A, (1 - np.repeat(A, d // gates, axis=1)) * X, [0, 3, rows], np.zeros((2, d)), reverse)
        _close("h", _f64(th), ref, E + U * (np.abs(ref) + E))
        da, dx = torch.empty((rows, gates), device="cuda"), torch.empty((rows, d), device="cuda")
        v.nerf_scan_grad(tdh, ta, tx, th, da, dx, offsets=off, reverse=reverse, mix=True)
        rda, rdx, _ = O.scan_grad(_f64(near[2]), None, A, X, _f64(th), None, [0, 3, rows], reverse, True)
        # (21 terms of at most four roundings each, gates of at most 1: a bound of the magnitudes' sum)
        m = np.abs(_f64(near[2])).sum(0)
        assert (np.abs(_f64(dx) - rdx) <= 8 * rows * U * 2 * m).all()
        top = np.abs(_f64(th)).max() + np.abs(X).max()
        assert (np.abs(_f64(da) - rda) <= 8 * (rows + d) * U * m.sum() * top).all()


@pytest.mark.parametrize("lens", [[5, 0, 40], [3000, 3, 5990], [4] * 300])
def test_rows_in_front_of_the_first_sequence(lens):
    """Rows before the first sequence and behind the last are left as they are."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"scan behind other rows {lens[:3]}")
    g = np.random.default_rng(len(lens))
    lead, d, n = 70, 20, len(lens)
    off = lead + _offsets(g, lens)
    rows = int(off[-1]) + 9
    a, x, h0 = _inputs(g, rows, d, d, n)
    ta, tx, th0 = _put(a, "f32"), _put(x, "f32"), _put(h0, "f32")
    a, x, h0 = _f64(ta), _f64(tx), _f64(th0)
    toff = torch.from_numpy(off.astype(np.int32)).cuda()
    h, da, dx = (torch.full((rows, d), 7.0, device="cuda") for _ in range(3))
    v.nerf_scan(ta, tx, h, h0=th0, offsets=toff)
    ref, _ = O.scan(a, x, off, h0)
    _, E, _ = _bounds(a, x, off, h0, False)
    inside = slice(lead, int(off[-1]))
    hh = _f64(h)
    _close("h", hh[inside], ref[inside], (E + U * (np.abs(ref) + E))[inside])
    v.nerf_scan_grad(tx, ta, None, h, da, dx, h0=th0, offsets=toff)
    _, rdx, _ = O.scan_grad(x, None, a, x, np.nan_to_num(hh), h0, off)
    _, E, _ = _bounds(a, a * x, off, np.zeros((n, d)), True)
    before = np.zeros((rows, d))  # errors of what flows into each row
    M, _, _ = _bounds(a, a * x, off, np.zeros((n, d)), True)
    mags = np.zeros((rows, d))
    for s in range(n):
        before[off[s]:max(off[s], off[s + 1] - 1)] = E[off[s] + 1:off[s + 1]]
        mags[off[s]:max(off[s], off[s + 1] - 1)] = M[off[s] + 1:off[s + 1]]
    tol = before + 2 * U * (np.abs(x) + mags)
    _close("dx", _f64(dx)[inside], rdx[inside], tol[inside])
    for t in (h, da, dx):
        assert (t[:lead] == 7.0).all() and (t[int(off[-1]):] == 7.0).all()


def test_two_split_calls_at_once():
    """Calls on two streams whose chunks wait for each other's neighbours only, results bit-equal to one at a time."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("two split scans at once")
    gen = torch.Generator(device="cuda").manual_seed(3)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda")
    jobs = []
    for rows, d in ((20000, 512), (30000, 128)):
        a, x = torch.sigmoid(mk(rows, d) + 3), mk(rows, d)
        want, dx, da = torch.empty_like(x), torch.empty_like(x), torch.empty_like(a)
        v.nerf_scan(a, x, want, mix=True)
        v.nerf_scan_grad(x, a, x, want, da, dx, mix=True)
        jobs.append((a, x, want, da, dx, [torch.empty_like(x) for _ in range(3)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        for a, x, want, da, dx, (h, da2, dx2), stream in jobs:
            with torch.cuda.stream(stream):
                v.nerf_scan(a, x, h, mix=True)
                v.nerf_scan_grad(x, a, x, h, da2, dx2, mix=True)
    torch.cuda.synchronize()
    for a, x, want, da, dx, (h, da2, dx2), _ in jobs:
        assert torch.equal(h, want) and torch.equal(da2, da) and torch.equal(dx2, dx)


def test_more_than_2_to_31_elements():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("scan of 2^31 elements and more")
    rows, d = (1 << 20) + 40, 2056
    x = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    x[-30:] = torch.randn((30, d), device="cuda").to(torch.bfloat16)
    a = torch.full((rows, 1), 0.5, device="cuda")
    h, last = torch.empty_like(x), torch.empty((1, d), device="cuda")
    v.nerf_scan(a, x, h, h_last=last)
    ref, rl = O.scan(np.full((30, 1), 0.5), _f64(x[-30:]), [0, 30])
    assert (np.abs(_f64(h[-30:]) - ref) <= 2.0 ** -7 * np.abs(ref) + 1e-6).all() and not h[:-30].any()
    assert np.allclose(_f64(last), rl, atol=1e-5)
    da, dx = torch.empty_like(a), torch.empty_like(x)
    v.nerf_scan_grad(x, a, None, h, da, dx)
    D = O.scan_grad(_f64(x[-30:]), None, np.full((30, 1), 0.5), None, _f64(h[-30:]), None, [0, 30])[1]
    assert (np.abs(_f64(dx[-30:]) - D) <= 2.0 ** -7 * np.abs(D) + 1e-6).all()
