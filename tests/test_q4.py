"""The 4-bit formats (levels -8..7, one fp16 scale per 32 or 128 weights) in every product
call, against the fp64 oracle.

Bounds, from the arithmetic. y is rounded once to bf16: half a step, 2^-8 |y| (none for
lbq_gemv_f32). fp32 sums: at most K / 16 + 8 additions one after another (a matrix
instruction adds 16 products at once), each off by at most 2^-23 of the sum of
magnitudes S = sum |w x|; with K <= 17408 that is below 2^-12 S. More than 16 tokens:
weights are rounded to fp16 before the product, 2^-11 of each term more.
"""
import ctypes
import os

import numpy as np
import pytest
import torch

from bit_weight_only_ternary_b200 import synth

Q4 = (5, 6)
GROUP = {5: 32, 6: 128}
NTHREADS = max(1, min(32, os.cpu_count() or 1))


@pytest.fixture(scope="module")
def L():
    from bit_weight_only_ternary_b200 import build
    build.build()
    from bit_weight_only_ternary_b200 import lbq
    return lbq


def _bound(Y, S, rounded=True, f16=False):
    return (2.0 ** -8 * np.abs(Y) if rounded else 0.0) + (2.0 ** -12 + (2.0 ** -11 if f16 else 0.0)) * S


def _inside(y, Y, S, what="", **kw):
    got = y.double().cpu().numpy().reshape(Y.shape)
    bad = ~(np.abs(got - Y) <= _bound(Y, S, **kw))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} out of bound, first {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]!r} for {Y[bad][0]!r}, S {S[bad][0]!r}")


def _make(L, orc, fmt, N, K, M, seed, scale_x=None):
    W = synth.weights(N, K, seed)
    X = synth.activations(M, K, seed + 1)
    if scale_x is not None:
        X = (X.double() * scale_x).to(torch.bfloat16)
    codes, scales = orc.pack(fmt, W.numpy())
    Y, S = orc.gemm(fmt, codes, scales, K, synth.bf16_bits(X), nthreads=NTHREADS)
    return L.lbq_pack(fmt, W.cuda()), X.cuda(), Y, S


# ------------------------------------------------------------------------------- CPU

@pytest.mark.parametrize("fmt", Q4)
def test_layout_matches_the_oracle(L, orc, fmt):
    for K in (128, 640, 5120, 17408):
        for N, N4 in ((3, 4), (4, 4), (9, 12)):
            ocs, oss, _ = orc.layout(fmt, K)
            assert L.lbq_packed_layout(fmt, K, N) == (ocs, oss, N4 * ocs, N4 * oss * 2)
            assert ocs == K // 2 and oss % 8 == 0 and oss >= K // GROUP[fmt]
    st = ctypes.c_int64()
    assert L.lib().lbq_packed_layout(fmt, 192, 4, ctypes.byref(st), None, None, None) == L.LBQ_ERR_SHAPE


@pytest.mark.parametrize("fmt", Q4)
def test_oracle_pack_against_numpy(orc, fmt):
    g, K, N = GROUP[fmt], 384, 6
    rng = np.random.default_rng(3)
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    W[1] = 0.0
    W[2] *= 1e9
    W[3] *= 1e-9
    W[4, :g] = np.tile(np.array([7, 0.5, 1.5, -0.5, -1.5, 2.5, -7, 3], np.float32), g // 8)  # ties
    codes, scales = orc.pack(fmt, W)
    blk = W.reshape(N, K // g, g).astype(np.float64)
    s = np.minimum(np.abs(blk).max(-1) / 7.0, 65504.0).astype(np.float16)
    assert np.array_equal(scales[:, :K // g], s.view(np.uint16))
    sd = s.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(sd > 0, np.clip(np.rint(blk / sd), -8, 7), 0.0).reshape(N, K).astype(int)
    words = codes.view("<u4")
    for i, nib in enumerate((0, 4, 1, 5, 2, 6, 3, 7)):  # the nibble of weight 8w + i
        assert np.array_equal((words >> (4 * nib)) & 15, (q[:, i::8] + 8).astype(np.uint32))
    t, bs = orc.unpack(fmt, codes, scales, K)
    assert np.array_equal(t, q) and np.array_equal(bs, s.astype(np.float64))
    assert np.array_equal(orc.dequant(fmt, codes, scales, K), q * np.repeat(s.astype(np.float64), g, 1))


def test_q4_refusals(L):
    lib = L.lib()
    x, y = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)

    def desc(fmt=5, K=512, N=4, codes=0x10000, scales=0x60000, cs=256, ss=16):
        return ctypes.byref(L.lbq_weights(fmt, 0, K, N, codes, scales, cs, ss))

    gemv = lambda d, xx=x, yy=y: lib.lbq_gemv(d, xx, None, yy, None, 0, None)  # noqa: E731
    assert gemv(desc(scales=None)) == L.LBQ_ERR_ARG
    assert gemv(desc(scales=0x60008)) == L.LBQ_ERR_ALIGN
    assert gemv(desc(ss=8)) == L.LBQ_ERR_SHAPE       # 512 / 32 scales a row
    assert gemv(desc(ss=20)) == L.LBQ_ERR_SHAPE
    assert gemv(desc(cs=240)) == L.LBQ_ERR_SHAPE
    assert gemv(desc(K=320)) == L.LBQ_ERR_SHAPE
    assert gemv(desc(N=0)) == L.LBQ_ERR_SHAPE
    assert gemv(desc(N=2 ** 28 + 1)) == L.LBQ_ERR_SHAPE
    assert gemv(desc(), ctypes.c_void_p(0x20008)) == L.LBQ_ERR_ALIGN
    assert gemv(desc(), x, ctypes.c_void_p(0x30001)) == L.LBQ_ERR_ALIGN
    assert lib.lbq_gemm(desc(), x, 0, None, y, None, 0, None) == L.LBQ_ERR_SHAPE
    ws = ctypes.c_void_p(0x40000)
    assert lib.lbq_gemv_f32(desc(), x, None, ctypes.c_void_p(0x30002), ws, 1 << 24, None) == L.LBQ_ERR_ALIGN
    need = lib.lbq_workspace_bytes(desc(), 1)
    assert need >= 65536 and gemv(desc()) == L.LBQ_ERR_WORKSPACE
    assert lib.lbq_gemv(desc(), x, None, y, ws, need - 1, None) == L.LBQ_ERR_WORKSPACE
    assert lib.lbq_gemv(desc(), x, None, y, ctypes.c_void_p(0x40008), need, None) == L.LBQ_ERR_ALIGN
    for M in (2, 16, 17, 300):
        need = lib.lbq_workspace_bytes(desc(), M)
        assert lib.lbq_gemm(desc(), x, M, None, y, ws, need - 1, None) == L.LBQ_ERR_WORKSPACE
    assert lib.lbq_gemv_noalloc(desc(scales=None), x, None, y, None) == L.LBQ_ERR_ARG
    W = ctypes.c_void_p(0x70000)
    assert lib.lbq_pack(5, W, 512, 4, ctypes.c_void_p(0x10000), None, None) == L.LBQ_ERR_ARG
    assert lib.lbq_pack(6, W, 500, 4, ctypes.c_void_p(0x10000), ctypes.c_void_p(0x60000), None) == L.LBQ_ERR_SHAPE
    arr = (L.lbq_product * 2)()
    for i in range(2):
        arr[i].w = L.lbq_weights(5, 0, 512, 4, 0x10000, 0x60000, 256, 16)
        arr[i].x, arr[i].D, arr[i].y = 0x20000, None, 0x30000 + 0x100 * i
    with pytest.raises(L.LbqError) as e:
        L.lbq_gemv_batch_plan(arr, 2, 4)
    assert e.value.status == L.LBQ_ERR_FORMAT
    arr[1].y = 0x20000  # an output over an input
    assert lib.lbq_gemv_batch(arr, 2, ctypes.c_void_p(0x40000), 1 << 20, None) == L.LBQ_ERR_ARG


# ------------------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("fmt", Q4)
@pytest.mark.parametrize("N,K", [(256, 512), (37, 1536), (1, 128), (9, 384), (6, 640)])
def test_pack_and_unpack_bit_exact(L, orc, fmt, N, K):
    W = synth.weights(N, K, 40 + N)
    g = GROUP[fmt]
    W[0] = 0.0
    if N > 5:
        W[1, :g] = torch.tensor([7, 0.5, 1.5, -0.5, -1.5, 2.5, -7, -0.0] * (g // 8))  # ties
        W[2] *= 1e9   # the scale saturates
        W[3] *= 1e-9  # subnormal scales
        W[4] *= 1e-12
    pw = L.lbq_pack(fmt, W.cuda())
    codes, scales = orc.pack(fmt, W.numpy())
    assert np.array_equal(pw.codes.cpu().numpy(), orc.group4(codes))
    assert np.array_equal(pw.scales.cpu().numpy().view(np.uint16), orc.group4(scales))
    t, s = L.lbq_unpack(pw)
    ot, osc = orc.unpack(fmt, codes, scales, K)
    assert np.array_equal(t.cpu().numpy(), ot) and np.array_equal(s.double().cpu().numpy(), osc)


SHAPES = [(1, 128), (5, 128), (31, 384), (33, 1152), (256, 512), (100, 4096), (7168, 5120), (129, 17408)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", Q4)
@pytest.mark.parametrize("N,K", SHAPES)
def test_gemv(L, orc, fmt, N, K):
    pw, X, Y, S = _make(L, orc, fmt, N, K, 1, 7 * N + K)
    y = torch.full((N + 2,), 7.0, dtype=torch.bfloat16, device="cuda")
    L.lbq_gemv(pw, X[0], y=y[:N])
    _inside(y[:N], Y[0], S[0], "gemv")
    assert (y[N:] == 7).all()
    _inside(L.lbq_gemv_f32(pw, X[0]), Y[0], S[0], "f32", rounded=False)
    assert torch.equal(L.lbq_gemv_noalloc(pw, X[0]), y[:N])
    assert torch.equal(L.lbq_gemv(pw, X[0]), y[:N])  # the same bits each time


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", Q4)
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 100, 130, 257])
@pytest.mark.parametrize("N,K", [(37, 640), (300, 1024)])
def test_gemm(L, orc, fmt, M, N, K):
    pw, X, Y, S = _make(L, orc, fmt, N, K, M, M + N + K)
    out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    L.lbq_gemm(pw, X, Y=out[:M])
    _inside(out[:M], Y, S, "gemm", f16=M > 16)
    assert (out[M] == 7).all()
    assert torch.equal(L.lbq_gemm(pw, X), out[:M])
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", Q4)
@pytest.mark.parametrize("M,N,K", [(24, 520, 5120), (300, 1000, 5120), (40, 65, 17408), (600, 128, 128)])
def test_gemm_larger(L, orc, fmt, M, N, K):
    pw, X, Y, S = _make(L, orc, fmt, N, K, M, M + N + K)
    _inside(L.lbq_gemm(pw, X), Y, S, "gemm", f16=True)
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", Q4)
@pytest.mark.parametrize("M", [1, 5, 40])
def test_activations_of_every_magnitude(L, orc, fmt, M):
    """Rows that span far more than fp16 does, rows that are tiny or huge, rows of zeros."""
    K = 640
    rng = torch.Generator().manual_seed(M)
    scale = torch.ones(M, K, dtype=torch.float64)
    scale[0] = 2.0 ** (torch.randint(-60, 61, (K,), generator=rng)).double()
    if M > 4:
        scale[1], scale[2], scale[3] = 2.0 ** -100, 2.0 ** 100, 0.0
    pw, X, Y, S = _make(L, orc, fmt, 70, K, M, 900 + M, scale_x=scale)
    got = L.lbq_gemm(pw, X)
    _inside(got, Y, S, "magnitudes", f16=M > 16)
    if M > 4:
        assert (got[3] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", Q4)
@pytest.mark.parametrize("M", [1, 3, 40])
def test_any_codes_scales_and_strides(L, orc, fmt, M):
    """Codes of another quantiser: every nibble, negative, zero, subnormal and the largest
    scales, rows with padding behind them."""
    N, K, g = 45, 384, GROUP[fmt]
    rng = np.random.default_rng(M)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    _, oss, _ = orc.layout(fmt, K)
    sc = (rng.standard_normal((N, oss)) * 0.01).astype(np.float16)
    sc[0], sc[1], sc[2] = 0.0, 65504.0, 6e-8
    scales = sc.view(np.uint16)
    X = synth.activations(M, K, 5)
    Y, S = orc.gemm(fmt, codes, scales, K, synth.bf16_bits(X))
    G = (N + 3) // 4
    cbuf = torch.full((G, 4 * (K // 2 + 32)), 0xA5, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((G, 4 * (oss + 8)), 0x7C01, dtype=torch.int16, device="cuda")  # a NaN behind each row
    cbuf[:, :2 * K] = torch.from_numpy(orc.group4(codes)).cuda()
    sbuf[:, :4 * oss] = torch.from_numpy(orc.group4(scales).view(np.int16)).cuda()
    pw = L.PackedWeights(fmt, K, N, cbuf, sbuf)
    got = L.lbq_gemm(pw, X.cuda()) if M > 1 else L.lbq_gemv(pw, X[0].cuda())
    # (a subnormal scale times a code is not off by more than fp16's smallest step)
    xa = np.abs(X.double().numpy()).sum(-1)[:, None]
    tiny = (2.0 ** -25 * xa) if M > 16 else 0.0
    err = np.abs(got.double().cpu().numpy().reshape(Y.shape) - Y)
    assert np.all(err <= _bound(Y, S, f16=M > 16) + tiny)
    z = got.reshape(M, N)[:, 0]
    assert (z == 0).all()


@pytest.mark.gpu
def test_batch_of_many_shapes_and_formats(L, orc):
    """A list of all formats and more products than one launch takes."""
    cases = [(5, 7168, 5120), (6, 5120, 17408), (5, 1, 128), (6, 45, 640), (1, 300, 512), (3, 70, 512)]
    cases += [(5 + i % 2, 1 + 13 * i % 90, 128 * (1 + i % 5)) for i in range(300)]
    items, want = [], []
    for i, (fmt, N, K) in enumerate(cases):
        W, x = synth.weights(N, K, 50 + i), synth.activations(1, K, 51 + i)
        codes, scales = orc.pack(fmt, W.numpy())
        Do = orc.rht_signs(9, K) if fmt == 3 else None
        Y, S = orc.gemm(fmt, codes, scales, K, synth.bf16_bits(x), Do, nthreads=NTHREADS)
        y = torch.full((N,), 5.0, dtype=torch.bfloat16, device="cuda")
        D = L.lbq_rht_signs(9, K) if fmt == 3 else None
        items.append((L.lbq_pack(fmt, W.cuda()), x[0].cuda(), D, y))
        want.append((Y[0], S[0]))
    plist = L.ProductList(items)
    ws = L.workspace_for_batch(plist)
    L.lbq_gemv_batch(plist, ws)
    first = [y.clone() for _, _, _, y in items]
    L.lbq_gemv_batch(plist, ws)
    assert all(torch.equal(y, f) for (_, _, _, y), f in zip(items, first))  # the same bits
    assert not ws[:65536].any()  # the counters are left at zero
    for (pw, x, D, y), (Y, S) in zip(items, want):
        if pw.fmt in Q4:
            # (sums may run in another order than in lbq_gemv, inside the same bound)
            _inside(y, Y, S, f"{pw.N}x{pw.K}")
        else:
            assert np.all(np.abs(y.double().cpu().numpy() - Y) <= 2.0 ** -8 * S)
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 12, 50])
def test_captured_replayed_and_on_another_stream(L, orc, M):
    """A chain of two products (the second reads the first's output) captured into a graph
    and replayed on new inputs, and the same on a side stream."""
    fmt, K, N = 5, 512, 384
    pa, X, _, _ = _make(L, orc, fmt, K, K, M, 60)
    pb, X2, _, _ = _make(L, orc, fmt, N, K, M, 62)
    h, y = torch.empty_like(X), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    wa, wb = L.workspace_for(pa, M), L.workspace_for(pb, M)

    def step(p, x, o, w):
        if M == 1:
            L.lbq_gemv(p, x[0], y=o[0], workspace=w)
        else:
            L.lbq_gemm(p, x, Y=o, workspace=w)

    def both():
        step(pa, X, h, wa)
        step(pb, h, y, wb)

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    X.copy_(X2)
    both()
    want = y.clone()
    y.fill_(9.0)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    y.fill_(9.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    assert torch.equal(y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", Q4)
@pytest.mark.parametrize("M,N,K", [(20, 40000, 256), (100, 40000, 384), (300, 30000, 128), (1000, 9000, 256)])
def test_many_tiles_for_every_pair_of_sms(L, fmt, M, N, K):
    """Products with several output tiles a pair of SMs, of up to 128 tokens and of more,
    with a few tokens that span more than fp16 holds (recomputed in fp32)."""
    W = torch.randn(N, K, generator=torch.Generator().manual_seed(3)).mul_(0.02).cuda()
    pw = L.lbq_pack(fmt, W)
    q, s = L.lbq_unpack(pw)
    dense = q.double() * s.double().repeat_interleave(K // s.shape[1], 1)
    X = synth.activations(M, K, 4)
    X[3, 5], X[M - 1, 7] = 2.0 ** 40, 2.0 ** -60
    X[M // 2] *= 2.0 ** -90
    X = X.cuda()
    Y = L.lbq_gemm(pw, X)
    assert torch.equal(Y, L.lbq_gemm(pw, X))
    x = X.double()
    want, S = x @ dense.t(), x.abs() @ dense.abs().t()
    err = (Y.double() - want).abs()
    lim = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12) * S
    assert (err <= lim).all(), f"worst {(err / lim).max()}"
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", Q4)
def test_tensor_parallel_shards(L, orc, fmt):
    """Shards of a matrix over three ranks: output rows beside one another, and input
    features whose fp32 partial products are summed."""
    from bit_weight_only_ternary_b200 import tp
    K, N, world = 1536, 300, 3
    W, X = synth.weights(N, K, 71), synth.activations(1, K, 72)
    codes, scales = orc.pack(fmt, W.numpy())
    Y, S = orc.gemm(fmt, codes, scales, K, synth.bf16_bits(X))
    x, pack = X[0].cuda(), lambda f, w: L.lbq_pack(f, w.cuda())
    col = torch.cat([tp.column_forward(tp.make_shard(W, fmt, "column", r, world, pack), x) for r in range(world)])
    _inside(col, Y[0], S[0], "column")
    part = torch.zeros(N, device="cuda")
    for r in range(world):
        s = tp.make_shard(W, fmt, "row", r, world, pack)
        part += L.lbq_gemv_f32(s.weights, x[s.lo:s.hi])
    _inside(part, Y[0], S[0], "row", rounded=False)


@pytest.mark.gpu
def test_offsets_past_32_bits(L):
    """Codes of more than 2^32 bytes (random ones, any code is a weight): the last rows."""
    fmt, g, K, N = 6, 128, 16384, 600_004
    cs, ss, _, _ = L.lbq_packed_layout(fmt, K, N)
    gen = torch.Generator("cuda").manual_seed(5)
    c = torch.randint(0, 256, (N // 4, 4 * cs), dtype=torch.uint8, device="cuda", generator=gen)
    assert c.numel() > 2 ** 32
    s = (torch.rand(N // 4, 4 * ss, device="cuda", generator=gen) * 0.01 + 0.001).half().view(torch.int16)
    pw = L.PackedWeights(fmt, K, N, c, s)
    q, sc = L.lbq_unpack(L.PackedWeights(fmt, K, 400, c[-100:].contiguous(), s[-100:].contiguous()))
    W = q.double() * sc.double().repeat_interleave(g, 1)
    for M in (1, 5, 40):
        X = synth.activations(M, K, 6).cuda()
        Y = L.lbq_gemv(pw, X[0])[None] if M == 1 else L.lbq_gemm(pw, X)
        want, S = X.double() @ W.t(), X.double().abs() @ W.abs().t()
        assert ((Y[:, -400:].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -12 + 2.0 ** -11) * S).all(), M
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", Q4)
@pytest.mark.parametrize("M", [1, 6, 40, 300])
@pytest.mark.parametrize("N", [64, 65])
def test_outputs_at_odd_addresses(L, orc, fmt, M, N):
    """Y two bytes off every wider boundary (K long enough to be split), nothing around it
    written."""
    K = 5120
    pw, X, Y, S = _make(L, orc, fmt, N, K, M, 81)
    buf = torch.full((M * N + 18,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[9:9 + M * N].view(M, N)
    if M == 1:
        L.lbq_gemv(pw, X[0], y=y[0])
    else:
        L.lbq_gemm(pw, X, Y=y)
    _inside(y, Y, S, "odd", f16=M > 8)
    assert (buf[:9] == 7).all() and (buf[9 + M * N:] == 7).all()
    z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(y, L.lbq_gemm(pw, X, Y=z) if M > 1 else L.lbq_gemv(pw, X[0], y=z[0])[None])
