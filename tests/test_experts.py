"""Slots sorted by expert, rows there and back with gradients, and the experts' products,
against plain 64-bit implementations.

Bounds, from the arithmetic: one bf16 rounding is half a step, 2^-8 of the value. A sum of
n fp32 terms is off by at most n 2^-23 of the sum of magnitudes S. The products' bounds
are those of the 4-bit products (test_q4.py): 2^-12 S for the sums, and 2^-11 S for fp16
weights where there are many rows an expert.
"""
import ctypes

import numpy as np
import pytest
import torch

from bit_weight_only_ternary_b200 import synth


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_ternary_b200 import build
    build.build()
    from bit_weight_only_ternary_b200 import lbq
    return lbq


def _sorted(ids, E):
    """offsets, rows, slots by plain Python."""
    flat = ids.reshape(-1).tolist()
    order = [i for e in range(E) for i in np.flatnonzero(np.asarray(flat) == e)]
    offsets = [0]
    for e in range(E):
        offsets.append(offsets[-1] + flat.count(e))
    rows = -np.ones(len(flat), np.int32)
    rows[order] = np.arange(len(order))
    slots = -np.ones(len(flat), np.int32)
    slots[:len(order)] = order
    return np.array(offsets, np.int32), rows.reshape(ids.shape), slots


def _ids(T, topk, E, seed, drop=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).pow(2).topk(min(topk, E), -1).indices.to(torch.int32)
    ids[torch.rand(ids.shape, generator=g) < drop] = -1
    return ids


# ------------------------------------------------------------------------------- CPU

def test_expert_refusals(L):
    lib = L.lib()
    p = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(8)]
    A, S, AL = L.LBQ_ERR_ARG, L.LBQ_ERR_SHAPE, L.LBQ_ERR_ALIGN
    odd = ctypes.c_void_p(0x100002)

    def sort(e=p[0], nb=4, T=4, k=2, E=8, o=p[1], r=p[2], s=p[3]):
        return lib.lbq_expert_sort(e, nb, T, k, E, o, r, s, None)
    assert sort(e=None) == A and sort(o=None) == A and sort(r=None) == A and sort(s=None) == A
    assert sort(nb=2) == A and sort(e=odd) == AL and sort(nb=8, e=ctypes.c_void_p(0x100004)) == AL
    assert sort(T=0) == S and sort(k=0) == S and sort(k=1025) == S and sort(E=0) == S and sort(E=1025) == S
    assert sort(T=2 ** 30, k=2) == S

    def disp(X=p[0], T=4, K=8, rows=p[1], k=2, w=None, R=8, out=p[2]):
        return lib.lbq_expert_dispatch(X, T, K, rows, k, w, R, out, None)
    assert disp(X=None) == A and disp(rows=None) == A and disp(out=None) == A and disp(out=p[0]) == A
    assert disp(T=0) == S and disp(K=0) == S and disp(R=0) == S and disp(K=2 ** 25) == S
    assert disp(X=ctypes.c_void_p(0x100001)) == AL and disp(rows=odd) == AL and disp(w=odd) == AL

    def comb(Y=p[0], R=8, N=8, rows=p[1], T=4, k=2, w=None, out=p[2]):
        return lib.lbq_expert_combine(Y, R, N, rows, T, k, w, out, None)
    assert comb(Y=None) == A and comb(rows=None) == A and comb(out=None) == A and comb(out=p[0]) == A
    assert comb(T=0) == S and comb(N=0) == S and comb(R=0) == S and comb(k=0) == S and comb(rows=odd) == AL

    def grad(d=p[0], Y=p[1], R=8, N=8, rows=p[2], T=4, k=2, w=p[3], dY=p[4], dw=p[5]):
        return lib.lbq_expert_combine_grad(d, Y, R, N, rows, T, k, w, dY, dw, None)
    for name in ("d", "Y", "rows", "w", "dY", "dw"):
        assert grad(**{name: None}) == A
    assert grad(dY=p[1]) == A and grad(dY=p[0]) == A and grad(dw=p[3]) == A
    assert grad(T=0) == S and grad(R=0) == S and grad(N=2 ** 25) == S and grad(dw=odd) == AL

    def prod(fmt=5, E=4, X=p[0], T=4, off=p[1], slots=p[2], k=2, R=8, Y=p[3], scales=0x900000, N=8):
        w = L.lbq_weights(fmt, 0, 512, N, 0x800000, scales, 256 if fmt == 5 else 112, 16 if fmt == 5 else 0)
        return lib.lbq_expert_gemm(ctypes.byref(w), E, X, T, off, slots, k, R, Y, None, 0, None)
    assert prod(fmt=1, scales=None) == L.LBQ_ERR_FORMAT and prod(fmt=4) == L.LBQ_ERR_FORMAT
    assert prod(X=None) == A and prod(off=None) == A and prod(Y=None) == A and prod(Y=p[0]) == A
    assert prod(E=0) == S and prod(E=1025) == S and prod(T=0) == S and prod(R=0) == S and prod(k=0) == S
    assert prod(slots=None) == S  # fewer input rows than output rows
    assert prod(X=ctypes.c_void_p(0x100008)) == AL and prod(slots=odd) == AL and prod(off=odd) == AL
    assert lib.lbq_expert_workspace_bytes(None, 4, 8) == 0


# ------------------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,topk,E,drop", [(1, 1, 1, 0), (1, 8, 128, 0), (3, 2, 4, 0.5), (33, 1, 1024, 0),
                                           (500, 8, 60, 0.1), (513, 8, 64, 0), (1000, 7, 1000, 0.3),
                                           (5000, 4, 9, 0.02), (64, 8, 16, 1.0)])
def test_sort(L, T, topk, E, drop, dtype):
    ids = _ids(T, topk, E, T + E, drop).to(dtype)
    if T > 30:
        ids[3, 0], ids[7, 0] = E, 2 ** 31 - 1  # out of range: left out
        if dtype == torch.int64:
            ids[9, 0] = 2 ** 40  # (its low 32 bits are 0)
    offsets, rows, slots = L.lbq_expert_sort(ids.cuda(), E)
    wo, wr, ws = _sorted(ids, E)
    assert np.array_equal(offsets.cpu(), wo) and np.array_equal(rows.cpu(), wr)
    assert np.array_equal(slots.cpu(), ws)


@pytest.mark.gpu
def test_sort_of_one_expert_and_repeated_choices(L):
    ids = torch.full((4097, 3), 5, dtype=torch.int32)  # one token names one expert three times
    offsets, rows, slots = L.lbq_expert_sort(ids.cuda(), 7)
    assert offsets.tolist() == [0] * 6 + [ids.numel()] * 2
    assert torch.equal(rows.view(-1).cpu(), torch.arange(ids.numel(), dtype=torch.int32))
    assert torch.equal(slots, rows.view(-1))


ROUTES = [(1, 1, 1, 8, 0), (1, 8, 16, 2048, 0), (7, 2, 8, 1001, 0.3), (130, 3, 5, 1, 0), (64, 11, 16, 4104, 0.5),
          (257, 8, 32, 520, 0.1)]


def _route(L, T, topk, E, drop, seed):
    ids = _ids(T, topk, E, seed, drop)
    offsets, rows, slots = L.lbq_expert_sort(ids.cuda(), E)
    return offsets, rows, slots, int(offsets[-1])


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("T,topk,E,N,drop", ROUTES)
def test_dispatch(L, T, topk, E, N, drop, shift):
    """(shift: rows that begin 2 bytes off a 16-byte boundary)"""
    _, rows, slots, kept = _route(L, T, topk, E, drop, 1)
    R = T * topk
    X = synth.activations(T, N, 2).cuda()
    Xs = torch.empty(T * N + 8, dtype=torch.bfloat16, device="cuda")[shift:shift + T * N].view(T, N).copy_(X)
    w = torch.rand(T, topk, device="cuda")
    tok = (slots[:kept] // topk).long()
    for weights in (None, w):
        out = torch.full((R + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
        L.lbq_expert_dispatch(Xs, rows, weights, out=out[:R])
        want = X.double()[tok]
        if weights is None:
            assert torch.equal(out[:kept].double(), want)
        else:
            want = want * w.double().view(-1)[slots[:kept].long()].unsqueeze(1)
            # the fp32 product and its bf16 rounding
            assert ((out[:kept].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs()).all()
        assert (out[kept:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,topk,E,N,drop", ROUTES)
def test_combine_and_its_gradients(L, T, topk, E, N, drop):
    offsets, rows, slots, kept = _route(L, T, topk, E, drop, 3)
    R = T * topk
    Y, dout = synth.activations(R, N, 4).cuda(), synth.activations(T, N, 5).cuda()
    Y[kept:] = float("nan")  # rows no slot names are not read
    w = torch.randn(T, topk, device="cuda")
    tok, slot = (slots[:kept] // topk).long(), slots[:kept].long()
    wd = w.double().view(-1)[slot].unsqueeze(1)
    for weights, ww in ((w, wd), (None, torch.ones_like(wd))):
        out = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
        L.lbq_expert_combine(Y, rows, weights, out=out[:T])
        terms = ww * Y[:kept].double()
        want = torch.zeros(T, N, dtype=torch.float64, device="cuda").index_add_(0, tok, terms)
        S = torch.zeros_like(want).index_add_(0, tok, terms.abs())
        assert ((out[:T].double() - want).abs() <= 2.0 ** -8 * want.abs() + topk * 2.0 ** -22 * S).all()
        assert (out[T] == 7).all()
    dY = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    dY, dw = L.lbq_expert_combine_grad(dout, Y, rows, w, dY=dY)
    want = wd * dout.double()[tok]
    assert ((dY[:kept].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs()).all()
    assert (dY[kept:] == 7).all()
    prod = dout.double()[tok] * Y[:kept].double()
    wantw = torch.zeros(R, dtype=torch.float64, device="cuda")
    wantw[slot] = prod.sum(1)
    Sw = torch.zeros_like(wantw)
    Sw[slot] = prod.abs().sum(1)
    assert ((dw.view(-1).double() - wantw).abs() <= N * 2.0 ** -23 * Sw).all()
    assert torch.equal(L.lbq_expert_combine_grad(dout, Y, rows, w, dY=dY)[1], dw)  # the same bits


@pytest.mark.gpu
def test_gradients_against_differences(L):
    """L(Y, w) = sum(dout * combine(Y, w)) is linear in each argument, so the difference
    between two points is the gradient times the step, up to the outputs' roundings."""
    T, topk, E, N = 5, 2, 4, 64
    _, rows, slots, kept = _route(L, T, topk, E, 0.0, 8)
    Y, dout = synth.activations(T * topk, N, 9).cuda(), synth.activations(T, N, 10).cuda()
    w = torch.rand(T, topk, device="cuda")
    dY, dw = L.lbq_expert_combine_grad(dout, Y, rows, w)
    dY = dY.double()

    def loss(Y, w):
        out = L.lbq_expert_combine(Y, rows, w).double()
        return (out * dout.double()).sum().item(), (2.0 ** -8 * out * dout.double()).abs().sum().item()
    base, r0 = loss(Y, w)
    for t in range(T):
        step = torch.zeros_like(w)
        step[t, 1] = 8.0
        l1, r1 = loss(Y, w + step)
        assert abs((l1 - base) - 8.0 * dw[t, 1].item()) <= 1.01 * (r0 + r1)
    for r in range(T * topk):
        Z = Y.clone()
        Z[r] = -Y[r]  # a step of -2 Y[r]
        l1, r1 = loss(Z, w)
        want = (dY[r] * (-2.0 * Y[r].double())).sum().item()
        slack = (2.0 ** -8 * dY[r] * 2.0 * Y[r].double()).abs().sum().item()
        assert abs((l1 - base) - want) <= 1.01 * (r0 + r1 + slack)


@pytest.mark.gpu
def test_rows_outside_the_buffer_are_left_out(L):
    T, N, R = 6, 16, 4
    rows = torch.tensor([[0], [-5], [3], [4], [2 ** 31 - 1], [1]], dtype=torch.int32, device="cuda")
    X = synth.activations(T, N, 1).cuda()
    buf = torch.full((R + 4, N), 7.0, dtype=torch.bfloat16, device="cuda")
    L.lbq_expert_dispatch(X, rows, out=buf[:R])
    assert torch.equal(buf[[0, 3, 1]], X[[0, 2, 5]]) and (buf[2] == 7).all() and (buf[R:] == 7).all()
    out = L.lbq_expert_combine(buf[:R].contiguous(), rows)
    assert torch.equal(out[[0, 2, 5]], X[[0, 2, 5]]) and (out[[1, 3, 4]] == 0).all()


def _experts(L, orc, fmt, E, N, K, seed):
    W = torch.stack([synth.weights(N, K, seed + e) for e in range(E)])
    ew = L.pack_experts(fmt, W.cuda())
    dense = torch.stack([torch.from_numpy(orc.dequant(fmt, *orc.pack(fmt, W[e].numpy()), K)) for e in range(E)])
    return ew, dense.cuda()


def _check_rows(Y, want, S, f16):
    err = (Y.double() - want).abs()
    lim = 2.0 ** -8 * want.abs() + (2.0 ** -12 + (2.0 ** -11 if f16 else 0)) * S
    assert (err <= lim).all(), f"{(err > lim).sum()} out of bound, worst {(err / lim).max()}"


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [5, 6])
@pytest.mark.parametrize("T,topk,E,N,K,drop", [(1, 1, 1, 5, 128, 0), (3, 2, 8, 70, 256, 0), (40, 4, 6, 33, 640, 0.2),
                                               (200, 2, 3, 130, 384, 0), (64, 8, 64, 256, 1024, 0),
                                               (700, 4, 5, 300, 512, 0.1), (9, 2, 4, 64, 256, 1.0)])
def test_expert_gemm(L, orc, fmt, T, topk, E, N, K, drop):
    ew, dense = _experts(L, orc, fmt, E, N, K, 30)
    offsets, rows, slots, kept = _route(L, T, topk, E, drop, T)
    R = T * topk
    X = synth.activations(T, K, 11).cuda()
    Y = torch.full((R + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=topk, Y=Y[:R])
    tok = (slots[:kept] // topk).long()
    e_of = torch.repeat_interleave(torch.arange(E, device="cuda"), (offsets[1:] - offsets[:-1]).long())
    want = torch.zeros(kept, N, dtype=torch.float64, device="cuda")
    S = torch.zeros_like(want)
    for e in range(E):
        m = e_of == e
        want[m] = X[tok[m]].double() @ dense[e].t()
        S[m] = X[tok[m]].double().abs() @ dense[e].abs().t()
    _check_rows(Y[:kept], want, S, True)
    assert (Y[kept:] == 7).all()
    # rows already in sorted order: the same bits
    xs = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    L.lbq_expert_dispatch(X, rows, out=xs)
    assert torch.equal(L.lbq_expert_gemm(ew, xs, offsets)[:kept], Y[:kept])
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [8, 400])
def test_bad_slots_and_offsets_stay_inside(L, orc, T):
    """Slots of no token give rows of zeros, offsets are clamped to the rows."""
    E, N, K = 3, 40, 256
    ew, dense = _experts(L, orc, 5, E, N, K, 90)
    X = synth.activations(T, K, 3).cuda()
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    slots[1], slots[2], slots[3] = -7, T, 2 ** 31 - 1
    offsets = torch.tensor([-4, T // 2, T // 2, T + 100], dtype=torch.int32, device="cuda")
    buf = torch.full((T + 8, N), 7.0, dtype=torch.bfloat16, device="cuda")
    L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=1, Y=buf[:T])
    assert (buf[T:] == 7).all() and (buf[1:4] == 0).all()
    want = torch.cat([X[:T // 2].double() @ dense[0].t(), X[T // 2:].double() @ dense[2].t()])
    S = torch.cat([X[:T // 2].double().abs() @ dense[0].abs().t(), X[T // 2:].double().abs() @ dense[2].abs().t()])
    keep = [0] + list(range(4, T))
    _check_rows(buf[keep], want[keep], S[keep], True)
    offsets.copy_(torch.tensor([T, 2, 1, 0]))  # nothing in order: no row
    buf.fill_(7.0)
    L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=1, Y=buf[:T])
    torch.cuda.synchronize()
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [5, 6])
@pytest.mark.parametrize("T,drop", [(1, 0.0), (6, 0.3), (300, 0.1)])
def test_a_layer_of_experts_eager_and_captured(L, orc, fmt, T, drop):
    """Sort, up product with the gather, activation, down product, combine: as one layer
    uses them, against 64 bits, then captured into a graph and replayed on other tokens."""
    E, topk, H, F = 12, 3, 256, 384
    up, Wu = _experts(L, orc, fmt, E, F, H, 200)
    down, Wd = _experts(L, orc, fmt, E, H, F, 300)
    R = T * topk
    X = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(T, topk, dtype=torch.int32, device="cuda")
    w = torch.empty(T, topk, device="cuda")
    bufs = {}

    def load(seed):
        X.copy_(synth.activations(T, H, seed))
        ids.copy_(_ids(T, topk, E, seed, drop))
        w.copy_(torch.rand(T, topk, generator=torch.Generator().manual_seed(seed)))

    wsu, wsd = L.workspace_for_experts(up, R), L.workspace_for_experts(down, R)

    def layer():
        offsets, rows, slots = L.lbq_expert_sort(ids, E)
        h = L.lbq_expert_gemm(up, X, offsets, slots=slots, topk=topk, workspace=wsu)
        bufs["h"] = h.clamp_(min=0)
        y = L.lbq_expert_gemm(down, bufs["h"], offsets, workspace=wsd)
        bufs["out"] = L.lbq_expert_combine(y, rows, w)
        bufs["rows"] = rows

    def check():
        h, rows = bufs["h"].double(), bufs["rows"]
        want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        lim = torch.zeros_like(want)
        for t in range(T):
            for j in range(topk):
                r, e = int(rows[t, j]), int(ids[t, j])
                if e < 0:
                    assert r == -1
                    continue
                # each step from the values the step before it gave: the up product ...
                z, S = Wu[e] @ X[t].double(), Wu[e].abs() @ X[t].double().abs()
                assert ((h[r] - z.clamp(min=0)).abs() <= 2.0 ** -8 * z.abs() + 2.0 ** -10 * S).all()
                # ... and the down product and the sum
                y, S = Wd[e] @ h[r], Wd[e].abs() @ h[r].abs()
                want[t] += w[t, j].double() * y
                lim[t] += w[t, j].double() * (2.0 ** -8 * y.abs() + 2.0 ** -10 * S)
        assert ((bufs["out"].double() - want).abs() <= 1.01 * lim + 2.0 ** -8 * want.abs()).all()

    load(1)
    layer()
    check()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for seed in (2, 3):
        load(seed)
        g.replay()
        torch.cuda.synchronize()
        check()
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
def test_python_refuses_what_the_c_call_cannot_see(L):
    X = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for bad in (lambda: L.lbq_expert_dispatch(X.float(), rows), lambda: L.lbq_expert_dispatch(X, rows.long()),
                lambda: L.lbq_expert_dispatch(X[:, ::2], rows), lambda: L.lbq_expert_dispatch(X, rows[:3]),
                lambda: L.lbq_expert_combine(X, rows, torch.zeros(4, 3, device="cuda")),
                lambda: L.lbq_expert_combine(X.cpu(), rows), lambda: L.lbq_expert_sort(rows.float(), 4)):
        with pytest.raises(L.LbqError):
            bad()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [8, 400])
def test_descending_offsets_compute_no_row(L, orc, T):
    """Ranges that would overlap (the rows 0 .. T of two experts) are not computed at all."""
    E, N, K = 3, 40, 256
    ew, _ = _experts(L, orc, 6, E, N, K, 91)
    X = synth.activations(T, K, 3).cuda()
    Y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    for off in ([0, T, 0, T], [0, T, T, T - 1], [T // 2, T // 4, T, T]):
        L.lbq_expert_gemm(ew, X, torch.tensor(off, dtype=torch.int32, device="cuda"), Y=Y)
        assert (Y == 7).all(), off
    L.lbq_expert_gemm(ew, X, torch.tensor([1, 1, T - 1, T - 1], dtype=torch.int32, device="cuda"), Y=Y)
    assert (Y[0] == 7).all() and (Y[T - 1] == 7).all() and not (Y[1:T - 1] == 7).all(1).any()
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
def test_weights_or_workspace_on_the_host_are_refused(L, orc):
    import dataclasses
    E, N, K, T = 2, 8, 128, 4
    ew, _ = _experts(L, orc, 6, E, N, K, 92)
    X = synth.activations(T, K, 3).cuda()
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    ws = L.workspace_for_experts(ew, T)
    for e, w in ((dataclasses.replace(ew, codes=ew.codes.cpu()), ws), (ew, ws.cpu())):
        with pytest.raises(L.LbqError):
            L.lbq_expert_gemm(e, X, off, workspace=w)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 200])
def test_values_that_are_not_finite_stay_in_their_rows(L, orc, T):
    """A token with NaN or infinities makes its own rows so, and no other: in the experts'
    products, and in the sums over rows."""
    E, topk, N, K = 4, 2, 70, 384
    ew, dense = _experts(L, orc, 5, E, N, K, 93)
    X = synth.activations(T, K, 4).cuda()
    ids = _ids(T, topk, E, 5, 0.0).cuda()
    offsets, rows, slots = L.lbq_expert_sort(ids, E)
    good = L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=topk)
    X[1, 7], X[2, 100] = float("nan"), float("inf")
    bad = L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=topk)
    hit = torch.zeros(T * topk, dtype=torch.bool, device="cuda")
    hit[rows[1].long()] = True
    assert bad[hit].isnan().all()
    for j in range(topk):  # infinity times a weight of zero is NaN, else infinity
        w = dense[int(ids[2, j])][:, 100]
        y = bad[rows[2, j]].float()
        assert torch.equal(y.isnan(), w == 0) and torch.equal(y[w != 0], torch.sign(w[w != 0]).float() * float("inf"))
    hit[rows[2].long()] = True
    assert torch.equal(bad[~hit], good[~hit])
    out = L.lbq_expert_combine(bad, rows)
    keep = [t for t in range(T) if t not in (1, 2)]
    assert out[keep].isfinite().all() and out[1].isnan().all()
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [6, 300])
def test_two_streams_and_two_graphs_at_once(L, orc, T):
    """Two layers' products in flight together, each with its own workspace, eager and as
    graphs captured apart, give what they give alone."""
    E, topk, N, K = 8, 2, 200, 512
    ids = _ids(T, topk, E, 6, 0.1).cuda()
    offsets, rows, slots = L.lbq_expert_sort(ids, E)
    kept = int(offsets[-1])
    sets = []
    for i in range(2):
        ew, _ = _experts(L, orc, 5 + i, E, N, K, 94 + i)
        X = synth.activations(T, K, 7 + i).cuda()
        Y = torch.zeros(T * topk, N, dtype=torch.bfloat16, device="cuda")
        ws = L.workspace_for_experts(ew, T * topk)
        sets.append((ew, X, Y, ws, L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=topk)[:kept].clone()))
    torch.cuda.synchronize()

    def run(i):
        ew, X, Y, ws, _ = sets[i]
        L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=topk, Y=Y, workspace=ws)

    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(i)
        graphs.append(g)
    for play in (run, lambda i: graphs[i].replay()):
        for s in sets:
            s[2].zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    play(i)
        torch.cuda.synchronize()
        for s in sets:
            assert torch.equal(s[2][:kept], s[4])
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,T,topk,E,N,K,skew", [(5, 1500, 2, 40, 1200, 384, 3.0), (6, 1500, 2, 40, 1200, 256, 1.0),
                                                   (5, 4000, 1, 9, 2500, 128, 6.0), (6, 300, 8, 200, 600, 128, 0.0)])
def test_experts_of_very_different_sizes(L, orc, fmt, T, topk, E, N, K, skew):
    """Several tiles for every pair of SMs, large and small ones and experts without rows."""
    ew = L.pack_experts(fmt, (torch.randn(E, N, K, generator=torch.Generator().manual_seed(8)) * 0.02).cuda())
    X = synth.activations(T, K, 9).cuda()
    g = torch.Generator().manual_seed(10)
    score = torch.rand(T, E, generator=g).log() / torch.linspace(1, 8, E).pow(skew)
    score[:, E // 2] = float("-inf")
    ids = score.topk(topk, -1).indices.to(torch.int32).cuda()
    offsets, rows, slots = L.lbq_expert_sort(ids, E)
    off = offsets.tolist()
    assert off[E] == T * topk and off[E // 2] == off[E // 2 + 1]
    Y = L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=topk)
    again = L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=topk)
    assert torch.equal(Y, again)
    for e in range(E):
        if off[e] == off[e + 1]:
            continue
        one = L.PackedWeights(fmt, K, N, ew.codes[e], ew.scales[e])
        q, s = L.lbq_unpack(one)
        W = q.double() * s.double().repeat_interleave(K // s.shape[1], 1)
        x = X[(slots[off[e]:off[e + 1]] // topk).long()].double()
        _check_rows(Y[off[e]:off[e + 1]], x @ W.t(), x.abs() @ W.abs().t(), True)
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("topk", [3, 11])
@pytest.mark.parametrize("N", [64, 77])
def test_weights_of_slots_left_out_do_not_count(L, topk, N):
    """A slot without a row adds nothing and has no gradient, whatever its weight is."""
    T, R = 9, 40
    g = torch.Generator().manual_seed(11)
    Y = torch.randn(R, N, generator=g).to(torch.bfloat16).cuda()
    dout = torch.randn(T, N, generator=g).to(torch.bfloat16).cuda()
    rows = torch.randperm(T * topk, generator=g).view(T, topk).to(torch.int32)
    rows[rows >= R] = -1
    rows[2] = -1
    rows[3, 0] = R
    w = torch.rand(T, topk, generator=g)
    keep = (rows >= 0) & (rows < R)
    clean = torch.where(keep, w, torch.zeros(()))
    bad = torch.where(keep, w, torch.tensor([float("nan"), float("inf")])[torch.arange(topk) % 2].expand(T, topk))
    rows, bad, clean = rows.cuda(), bad.cuda().contiguous(), clean.cuda()
    out = L.lbq_expert_combine(Y, rows, bad)
    assert out.isfinite().all() and (out[2] == 0).all()
    assert torch.equal(out, L.lbq_expert_combine(Y, rows, clean))
    dY, dw = L.lbq_expert_combine_grad(dout, Y, rows, bad, dY=torch.zeros_like(Y))
    assert dY.isfinite().all() and dw.isfinite().all() and (dw.cpu()[~keep] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [5, 6])
@pytest.mark.parametrize("E,T,topk", [(1000, 40, 2), (1024, 1, 5), (513, 600, 3), (700, 3000, 4)])
def test_as_many_experts_as_there_may_be(L, fmt, E, T, topk):
    """More experts than threads, most or none of them without rows."""
    N, K = 9, 128
    ew = L.pack_experts(fmt, (torch.randn(E, N, K, generator=torch.Generator().manual_seed(12)) * 0.02).cuda())
    X = synth.activations(T, K, 13).cuda()
    ids = _ids(T, topk, E, 14, 0.05).cuda()
    offsets, rows, slots = L.lbq_expert_sort(ids, E)
    Y = L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=topk)
    one = [L.lbq_unpack(L.PackedWeights(fmt, K, N, ew.codes[e], ew.scales[e])) for e in range(E)]
    W = torch.stack([a.double() * b.double().repeat_interleave(K // b.shape[1], 1) for a, b in one])
    r, e = rows.flatten().long(), ids.flatten().long()
    keep = e >= 0
    x = X.double().repeat_interleave(topk, 0)[keep]
    want = torch.einsum("rnk,rk->rn", W[e[keep]], x)
    S = torch.einsum("rnk,rk->rn", W[e[keep]].abs(), x.abs())
    _check_rows(Y[r[keep]], want, S, True)
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
def test_expert_offsets_past_32_bits(L):
    """The last expert of matrices of more than 2^32 bytes (random codes)."""
    fmt, g, E, N, K = 5, 32, 64, 9600, 16384
    cs, ss, _, _ = L.lbq_packed_layout(fmt, K, N)
    gen = torch.Generator("cuda").manual_seed(5)
    c = torch.randint(0, 256, (E, N // 4, 4 * cs), dtype=torch.uint8, device="cuda", generator=gen)
    assert c.numel() > 2 ** 32
    s = (torch.rand(E, N // 4, 4 * ss, device="cuda", generator=gen) * 0.01 + 0.001).half().view(torch.int16)
    ew = L.ExpertWeights(fmt, K, N, E, c, s)
    q, sc = L.lbq_unpack(L.PackedWeights(fmt, K, N, c[-1], s[-1]))
    W = q.double() * sc.double().repeat_interleave(g, 1)
    for T in (8, 700):
        X = synth.activations(T, K, 6).cuda()
        ids = _ids(T, 2, E, 7).cuda()
        ids[0, 0] = ids[T - 1, 1] = E - 1
        offsets, rows, slots = L.lbq_expert_sort(ids, E)
        Y = L.lbq_expert_gemm(ew, X, offsets, slots=slots, topk=2)
        a = int(offsets[E - 1])
        x = X[(slots[a:] // 2).long()].double()
        _check_rows(Y[a:], x @ W.t(), x.abs() @ W.abs().t(), True)
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
def test_rows_past_32_bits(L):
    """More than 2^31 values in the rows' buffers."""
    T, topk, N, E = 33000, 8, 8192, 16
    part = torch.randn(1000, N, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    Y = part.repeat(T * topk // 1000, 1)
    assert Y.numel() > 2 ** 31
    ids = torch.randint(0, E, (T, topk), generator=torch.Generator().manual_seed(9)).cuda()
    offsets, rows, slots = L.lbq_expert_sort(ids, E)
    assert torch.equal(slots.long(), torch.argsort(ids.flatten(), stable=True))
    w = torch.rand(T, topk, generator=torch.Generator().manual_seed(10)).cuda()
    out = L.lbq_expert_combine(Y, rows, w)
    dY, dw = L.lbq_expert_combine_grad(out, Y, rows, w)
    last = int(slots[-1]) // topk  # the token of the last row
    for t in (0, last, T - 1):
        y, o, c = Y[rows[t].long()].double(), out[t].double(), w[t].double()[:, None]
        want = (c * y).sum(0)
        assert ((o - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * (c * y.abs()).sum(0)).all()
        # fp32 sums of 8192 products in a tree of short sums: far below 2^-16 of their magnitudes
        assert ((dw[t].double() - y @ o).abs() <= 2.0 ** -16 * (y.abs() @ o.abs())).all()
        assert ((dY[rows[t].long()].double() - c * o).abs() <= 2.0 ** -8 * (c * o).abs()).all()
    del dY, Y
    x = L.lbq_expert_dispatch(out, rows)
    assert torch.equal(x[-1], out[last]) and torch.equal(x[rows[T - 1].long()], out[T - 1].expand(topk, N))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 90])
def test_a_chain_of_every_kind_of_call(L, T):
    """Ternary, 4-bit and expert calls, each reading what the one before wrote, enqueued
    without a pause: the bits of the same calls with a wait after each (the kernels start
    early beside their predecessors)."""
    H, F, E, topk = 512, 1024, 16, 3
    g = torch.Generator().manual_seed(15)
    rnd = lambda *s: (torch.randn(*s, generator=g) * 0.05).cuda()
    tern, q4a, q4b = L.lbq_pack(1, rnd(H, H)), L.lbq_pack(5, rnd(F, H)), L.lbq_pack(6, rnd(H, F))
    up, down = L.pack_experts(6, rnd(E, F, H)), L.pack_experts(5, rnd(E, H, F))
    X0 = synth.activations(T, H, 16).cuda()
    idss = [_ids(T, topk, E, 17 + i, 0.1).cuda() for i in range(8)]
    w = torch.rand(T, topk, generator=g).cuda()
    R = T * topk
    new = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    ws = {id(p): L.workspace_for(p, T) for p in (tern, q4a, q4b)}
    wse = {id(p): L.workspace_for_experts(p, R) for p in (up, down)}
    a, b, c, h, y, x = new(T, H), new(T, F), new(T, H), new(R, F), new(R, H), new(T, H)
    off, rows, slots = new(E + 1, dt=torch.int32), new(T, topk, dt=torch.int32), new(R, dt=torch.int32)

    def product(p, src, dst):
        if T == 1:
            L.lbq_gemv(p, src[0], y=dst[0], workspace=ws[id(p)])
        else:
            L.lbq_gemm(p, src, Y=dst, workspace=ws[id(p)])

    def run(wait):
        x.copy_(X0)
        for ids in idss:
            for step in (lambda: product(tern, x, a), lambda: product(q4a, a, b), lambda: product(q4b, b, c),
                         lambda: L.lbq_expert_sort(ids, E, off, rows, slots),
                         lambda: L.lbq_expert_gemm(up, c, off, slots=slots, topk=topk, Y=h, workspace=wse[id(up)]),
                         lambda: L.lbq_expert_gemm(down, h, off, Y=y, workspace=wse[id(down)]),
                         lambda: L.lbq_expert_combine(y, rows, w, out=x),
                         lambda: L.lbq_expert_dispatch(x, rows, out=y),
                         lambda: L.lbq_expert_combine(y, rows, None, out=x)):
                step()
                if wait:
                    torch.cuda.synchronize()
            x.mul_(0.25 * X0.float().norm() / x.float().norm())
        return x.clone()

    want = run(True)
    assert want.isfinite().all() and want.float().norm() > 0
    for _ in range(10):
        assert torch.equal(run(False), want)
    assert L.lbq_device_fault() == 0
