"""Rows, weights, streams and buffers at the edges of what the 4-bit and expert calls take.

Bounds as in test_q4.py: one bf16 rounding is 2^-8 of the value; fp32 sums are within
2^-12 of the sum of magnitudes S; weights rounded to fp16 (many rows, on the tensor cores)
add 2^-11 S.
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


def _us(f, n=8):
    """The fastest of n runs in us, on the device."""
    f()
    best = float("inf")
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
    return best


def _dense(L, pw):
    """The fp64 weights of a packed matrix."""
    q, s = L.lbq_unpack(pw)
    return q.double() * s.double().repeat_interleave(pw.K // s.shape[1], 1)


# ------------------------------------------------------- what a row of activations holds

@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 1, 6, 7])
@pytest.mark.parametrize("experts", [False, True])
def test_the_smallest_value_of_all_counts(L, at, experts):
    """A row of ones with one 2^-133 beside a zero, on weights that are zero everywhere but
    there: fp16 cannot hold both, so the row is recomputed in fp32."""
    K, N, M = 256, 40, 70
    q = torch.full((N, K), 8, dtype=torch.int32)
    q[:, at] = 15
    word = torch.zeros(N, K // 8, dtype=torch.int32)
    for i in range(8):
        word |= q[:, i::8] << (4 * ((i >> 1) + 4 * (i & 1)))
    codes = word.view(N // 4, 4, K // 8).transpose(1, 2).contiguous().view(torch.uint8).view(N // 4, 2 * K)
    scales = torch.full((N // 4, 32), 65504.0, dtype=torch.float16).view(torch.int16)
    X = torch.ones(M, K, dtype=torch.bfloat16)
    X[:, at ^ 1], X[:, at] = 0.0, 2.0 ** -133
    if experts:
        ew = L.ExpertWeights(5, K, N, 1, codes[None].cuda(), scales[None].cuda())
        Y = L.lbq_expert_gemm(ew, X.cuda(), torch.tensor([0, M], dtype=torch.int32, device="cuda"))
    else:
        Y = L.lbq_gemm(L.PackedWeights(5, K, N, codes.cuda(), scales.cuda()), X.cuda())
    want = 7 * 65504.0 * 2.0 ** -133  # (a normal bf16 value's range; exact in fp32)
    assert ((Y.double() - want).abs() <= 2.0 ** -8 * want).all(), Y[0, :2].tolist()
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("experts", [False, True])
def test_rows_of_zeros_take_no_longer(L, experts):
    """Padding tokens are ordinary rows (recomputed apart, they took 130 times as long)."""
    K, N, M, E = 2048, 2048, 1024, 4
    gen = torch.Generator("cuda").manual_seed(3)
    W = torch.randn(E if experts else 1, N, K, device="cuda", generator=gen) * 0.02
    X = torch.randn(M, K, device="cuda", generator=gen).to(torch.bfloat16)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    if experts:
        w = L.pack_experts(6, W)
        off = torch.arange(0, M + 1, M // E, dtype=torch.int32, device="cuda")
        ws = L.workspace_for_experts(w, M)
        run = lambda: L.lbq_expert_gemm(w, X, off, Y=Y, workspace=ws)  # noqa: E731
    else:
        w = L.lbq_pack(6, W[0])
        ws = L.workspace_for(w, M)
        run = lambda: L.lbq_gemm(w, X, Y=Y, workspace=ws)  # noqa: E731
    ordinary = _us(run)
    full = Y.clone()
    X[::2] = 0
    zeros = _us(run)
    assert (Y[::2] == 0).all() and torch.equal(Y[1::2], full[1::2])
    assert zeros <= 2 * ordinary, f"{zeros:.1f} us, {ordinary:.1f} without rows of zeros"


# --------------------------------------------------------------- the experts' weights

def _blank_experts(L, fmt, E, N, K, device="cpu"):
    cs, ss, _, _ = L.lbq_packed_layout(fmt, K, N)
    G = (N + 3) // 4
    return L.ExpertWeights(fmt, K, N, E, torch.zeros(E, G, 4 * cs, dtype=torch.uint8, device=device),
                           torch.zeros(E, G, 4 * ss, dtype=torch.int16, device=device))


@pytest.mark.parametrize("fmt", [5, 6])
def test_experts_that_do_not_lie_behind_one_another_are_refused(L, fmt):
    """The C call sees a pointer to expert 0 and sizes: a strided choice of experts, more
    experts than there are, or tensors of other shapes or types would be read elsewhere."""
    E, N, K = 6, 10, 256
    ew = _blank_experts(L, fmt, E, N, K)
    c, s = ew.codes, ew.scales
    make = lambda **kw: L.ExpertWeights(**{**dict(fmt=fmt, K=K, N=N, E=E, codes=c, scales=s), **kw})  # noqa: E731
    assert L.lbq_expert_workspace_bytes(ew, 8) > 0
    half = make(E=3, codes=c[::2].contiguous(), scales=s[::2].contiguous())
    assert L.lbq_expert_workspace_bytes(half, 8) > 0
    assert half.desc().code_stride == ew.desc().code_stride
    for kw, status in ((dict(E=3, codes=c[::2], scales=s[::2]), L.LBQ_ERR_ARG),
                       (dict(E=3, codes=c[::2].contiguous(), scales=s[::2]), L.LBQ_ERR_ARG),
                       (dict(E=7), L.LBQ_ERR_SHAPE), (dict(E=5), L.LBQ_ERR_SHAPE),
                       (dict(scales=s[:5]), L.LBQ_ERR_SHAPE), (dict(codes=c[:, 1:].contiguous()), L.LBQ_ERR_SHAPE),
                       (dict(N=14), L.LBQ_ERR_SHAPE), (dict(codes=c[0]), L.LBQ_ERR_SHAPE),
                       (dict(codes=c.short()), L.LBQ_ERR_ARG), (dict(scales=s.int()), L.LBQ_ERR_ARG),
                       (dict(codes=c[:, :, 1:].contiguous()), L.LBQ_ERR_SHAPE)):
        with pytest.raises(L.LbqError) as e:
            L.lbq_expert_workspace_bytes(make(**kw), 8)
        assert e.value.status == status, kw.keys()
    # one row group: whatever stride a dimension of one element claims
    one = _blank_experts(L, fmt, 1, 4, K)
    odd = L.ExpertWeights(fmt, K, 4, 1, one.codes.as_strided(one.codes.shape, (7, 5, 1)), one.scales)
    assert odd.desc().code_stride == one.desc().code_stride == K // 2


@pytest.mark.gpu
def test_scales_on_the_host_are_refused(L):
    import dataclasses
    ew = _blank_experts(L, 5, 2, 8, 128, "cuda")
    X = synth.activations(4, 128, 3).cuda()
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for bad in (dataclasses.replace(ew, scales=ew.scales.cpu()), dataclasses.replace(ew, codes=ew.codes.cpu()),
                dataclasses.replace(ew, E=3)):
        with pytest.raises(L.LbqError):
            L.lbq_expert_gemm(bad, X, off if bad.E == 2 else torch.zeros(bad.E + 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(L.LbqError):
        L.lbq_expert_gemm(ew, X, off, workspace=torch.zeros(1 << 20, 2, dtype=torch.uint8, device="cuda")[:, 0])
    assert (L.lbq_expert_gemm(ew, X, off) == 0).all()


# ----------------------------------------------------------------- streams and memory

@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_calls_on_a_side_stream_make_their_own_memory_there(L, raw):
    """stream= names another stream than torch's current one, which is busy: a workspace
    that the call makes is zeroed and used in that stream's order."""
    K, N, E, R = 5120, 320, 3, 9
    gen = torch.Generator("cuda").manual_seed(5)
    W = torch.randn(E, N, K, device="cuda", generator=gen) * 0.02
    X = torch.randn(R, K, device="cuda", generator=gen).to(torch.bfloat16)
    pw, ew = L.lbq_pack(5, W[0]), L.pack_experts(5, W)
    off = torch.tensor([0, 2, 5, R], dtype=torch.int32, device="cuda")
    ids = torch.tensor([[0, 2], [1, 2], [0, 1]], device="cuda")

    big = X.repeat(8, 1)
    plist = L.ProductList([(pw, X[i], None, torch.empty(N, dtype=torch.bfloat16, device="cuda")) for i in range(3)])

    def calls(stream):
        L.lbq_gemv_batch(plist, stream=stream)
        return [L.lbq_gemv(pw, X[0], stream=stream), L.lbq_gemv_f32(pw, X[1], stream=stream),
                L.lbq_gemm(pw, X, stream=stream), L.lbq_gemm(pw, big, stream=stream),
                L.lbq_expert_gemm(ew, X, off, stream=stream), L.lbq_gemv_noalloc(pw, X[2], stream=stream),
                *L.lbq_expert_sort(ids, E, stream=stream), *[i[3] for i in plist.items]]

    want = [t.clone() for t in calls(None)]
    side = torch.cuda.Stream()
    for _ in range(3):
        # blocks of the workspaces' sizes, full of ones, given back to the current stream's pool
        dirty = [torch.ones(n, dtype=torch.uint8, device="cuda") for n in (103424, 217088, 368640, 1 << 20) for _ in range(4)]
        for _, _, _, y in plist.items:
            y.fill_(7)
        torch.cuda.synchronize()
        del dirty
        torch.cuda._sleep(40_000_000)  # (some 20 ms)
        got = calls(side.cuda_stream if raw else side)
        side.synchronize()
        with torch.cuda.stream(side):
            assert [torch.equal(g, w) for g, w in zip(got, want)] == [True] * len(want)
        torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(calls(0), want))  # the default stream by its handle
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(5120, 5120), (17408, 33), (640, 4096)])
def test_tiles_that_several_ctas_share_join_alike_every_time(L, K, N):
    """One and five tokens, and the same matrix as an expert: 200 runs give the same bits
    (the last CTA of a tile reads the others' parts)."""
    gen = torch.Generator("cuda").manual_seed(6)
    W = torch.randn(1, N, K, device="cuda", generator=gen) * 0.02
    X = torch.randn(5, K, device="cuda", generator=gen).to(torch.bfloat16)
    pw, ew = L.lbq_pack(6, W[0]), L.pack_experts(6, W)
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    w1, w5, we = L.workspace_for(pw, 1), L.workspace_for(pw, 5), L.workspace_for_experts(ew, 5)
    runs = [lambda: L.lbq_gemv(pw, X[0], workspace=w1), lambda: L.lbq_gemm(pw, X, workspace=w5),
            lambda: L.lbq_expert_gemm(ew, X, off, workspace=we)]
    want = [r() for r in runs]
    dense = X.double() @ _dense(L, pw).t()
    S = X.double().abs() @ _dense(L, pw).abs().t()
    for w in (want[0][None], want[1], want[2]):
        assert ((w.double() - dense[:len(w)]).abs() <= 2.0 ** -8 * dense[:len(w)].abs() + 2.0 ** -12 * S[:len(w)]).all()
    for _ in range(200):
        assert all(torch.equal(r(), w) for r, w in zip(runs, want))
    assert not any(w[:65536].any() for w in (w1, w5, we))


class _KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.POINTER(ctypes.c_void_p)), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _noalloc_counters(pw, L, x, y):
    """The address of the fixed array's arrival counters, from the arguments of a captured
    lbq_gemv_noalloc: the product's parts lie 64 KB behind them."""
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        L.lbq_gemv_noalloc(pw, x, y=y)
    cu = ctypes.CDLL("libcuda.so.1")
    graph, n = ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t()
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    for node in nodes:
        kind, p = ctypes.c_int(), _KernelNode()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value != 0 or cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) != 0:
            continue
        if p.smem < 65536:  # (not the product)
            continue
        words = ctypes.cast(p.params[0], ctypes.POINTER(ctypes.c_uint64))[:8]
        for a, b in zip(words, words[1:]):
            if a - b == 65536:
                return b
    raise AssertionError("no product among the captured kernels")


@pytest.mark.gpu
def test_noalloc_after_calls_that_overlapped(L):
    """Calls that overlap on the fixed array are wrong themselves (documented), but may
    leave counts in it: the calls after them are right all the same."""
    K, N = 5120, 5120
    gen = torch.Generator("cuda").manual_seed(7)
    pw = L.lbq_pack(5, torch.randn(N, K, device="cuda", generator=gen) * 0.02)
    x = torch.randn(K, device="cuda", generator=gen).to(torch.bfloat16)
    want = L.lbq_gemv(pw, x)
    y = torch.empty_like(want)
    assert torch.equal(L.lbq_gemv_noalloc(pw, x, y=y), want)
    at = _noalloc_counters(pw, L, x, y)
    left = torch.ones(1024, dtype=torch.int32)
    for count in (1, 2, 7):
        torch.cuda.synchronize()
        left.fill_(count)
        assert ctypes.CDLL("libcuda.so.1").cuMemcpyHtoD_v2(ctypes.c_uint64(at), ctypes.c_void_p(left.data_ptr()),
                                                           ctypes.c_size_t(4 * left.numel())) == 0
        for _ in range(3):
            y.fill_(7)
            assert torch.equal(L.lbq_gemv_noalloc(pw, x, y=y), want)


# ------------------------------------------------------------------------- workspaces

@pytest.mark.parametrize("fmt", [5, 6])
@pytest.mark.parametrize("K,N", [(128, 4), (768, 2048), (512, 256), (5120, 7001), (17408, 300), (5120, 34816),
                                 (5120, 18944), (8192, 9472)])
def test_a_workspace_for_more_rows_serves_fewer(L, fmt, K, N):
    """No call of fewer rows needs more bytes than one of more."""
    lib = L.lib()
    cs, ss, _, _ = L.lbq_packed_layout(fmt, K, N)
    w = ctypes.byref(L.lbq_weights(fmt, 0, K, N, 1 << 20, 1 << 20, cs, ss))
    rows = [*range(1, 700), *range(701, 3000, 37), 4096, 8192, 20000]
    need = [lib.lbq_workspace_bytes(w, M) for M in rows]
    assert need[0] >= 65536 and all(a <= b for a, b in zip(need, need[1:]))
    for E in (1, 8, 128):
        need = [lib.lbq_expert_workspace_bytes(w, E, R) for R in rows]
        assert need[0] >= 65536 and all(a <= b for a, b in zip(need, need[1:]))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [5, 6])
def test_one_workspace_for_every_batch(L, fmt):
    """The largest batch's workspace in calls of every smaller size, K split or not, few rows
    or many, in turn."""
    K, N, E = 2048, 768, 8
    gen = torch.Generator("cuda").manual_seed(8)
    W = torch.randn(E, N, K, device="cuda", generator=gen) * 0.02
    X = torch.randn(300, K, device="cuda", generator=gen).to(torch.bfloat16)
    pw, ew = L.lbq_pack(fmt, W[0]), L.pack_experts(fmt, W)
    ws, we = L.workspace_for(pw, 300), L.workspace_for_experts(ew, 300)
    for M in (300, 5, 65, 64, 33, 32, 1, 9, 257, 8, 100):
        off = torch.linspace(0, M, E + 1).to(torch.int32).cuda()
        assert torch.equal(L.lbq_expert_gemm(ew, X[:M], off, workspace=we), L.lbq_expert_gemm(ew, X[:M], off))
        if M == 1:
            assert torch.equal(L.lbq_gemv(pw, X[0], workspace=ws), L.lbq_gemv(pw, X[0]))
        else:
            assert torch.equal(L.lbq_gemm(pw, X[:M], workspace=ws), L.lbq_gemm(pw, X[:M]))
    assert not ws[:65536].any() and not we[:65536].any()


# --------------------------------------------------- buffers that lie over one another

def test_outputs_over_anything_else_are_refused(L):
    """Addresses only: every call answers before a launch. In each, an output or the
    workspace reaches one byte into something else, or stands where it does."""
    lib, A = L.lib(), L.LBQ_ERR_ARG
    V = ctypes.c_void_p
    T, k, E, N, K, R = 6, 2, 4, 16, 256, 12
    G, cs, ss = N // 4, K // 2, 8
    size = {"ids": 8 * R, "off": 4 * (E + 1), "rows": 4 * R, "slots": 4 * R, "w": 4 * R, "X": 2 * T * K, "Xs": 2 * R * K,
            "Y": 2 * R * N, "out": 2 * T * N, "dY": 2 * R * N, "dw": 4 * R, "codes": E * G * 4 * cs,
            "scales": E * G * 4 * ss * 2, "y1": 2 * N, "y32": 4 * N, "x1": 2 * K, "Ym": 2 * T * N}
    desc = lambda a, e=1: ctypes.byref(L.lbq_weights(5, 0, K, N, a["codes"], a["scales"], cs, ss))  # noqa: E731
    some = desc({"codes": 1 << 20, "scales": 1 << 20})
    size["ws1"], size["wsm"] = lib.lbq_workspace_bytes(some, 1), lib.lbq_workspace_bytes(some, T)
    size["wse"] = lib.lbq_expert_workspace_bytes(some, E, R)
    size["c1"], size["s1"] = G * 4 * cs, G * 4 * ss * 2
    place = {n: (i + 1) << 24 for i, n in enumerate(size)}
    calls = {  # written, read, the call
        "sort": (("off", "rows", "slots"), ("ids",),
                 lambda a: lib.lbq_expert_sort(V(a["ids"]), 8, T, k, E, V(a["off"]), V(a["rows"]), V(a["slots"]), None)),
        "dispatch": (("Xs",), ("X", "rows", "w"),
                     lambda a: lib.lbq_expert_dispatch(V(a["X"]), T, K, V(a["rows"]), k, V(a["w"]), R, V(a["Xs"]), None)),
        "combine": (("out",), ("Y", "rows", "w"),
                    lambda a: lib.lbq_expert_combine(V(a["Y"]), R, N, V(a["rows"]), T, k, V(a["w"]), V(a["out"]), None)),
        "grad": (("dY", "dw"), ("out", "Y", "rows", "w"),
                 lambda a: lib.lbq_expert_combine_grad(V(a["out"]), V(a["Y"]), R, N, V(a["rows"]), T, k, V(a["w"]), V(a["dY"]),
                                                       V(a["dw"]), None)),
        "experts": (("Y", "wse"), ("X", "off", "slots", "codes", "scales"),
                    lambda a: lib.lbq_expert_gemm(desc(a), E, V(a["X"]), T, V(a["off"]), V(a["slots"]), k, R, V(a["Y"]),
                                                  V(a["wse"]), size["wse"], None)),
        "gemv": (("y1", "ws1"), ("x1", "c1", "s1"),
                 lambda a: lib.lbq_gemv(desc({"codes": a["c1"], "scales": a["s1"]}), V(a["x1"]), None, V(a["y1"]), V(a["ws1"]),
                                        size["ws1"], None)),
        "gemv_f32": (("y32", "ws1"), ("x1", "c1", "s1"),
                     lambda a: lib.lbq_gemv_f32(desc({"codes": a["c1"], "scales": a["s1"]}), V(a["x1"]), None, V(a["y32"]),
                                                V(a["ws1"]), size["ws1"], None)),
        "gemm": (("Ym", "wsm"), ("X", "c1", "s1"),
                 lambda a: lib.lbq_gemm(desc({"codes": a["c1"], "scales": a["s1"]}), V(a["X"]), T, None, V(a["Ym"]), V(a["wsm"]),
                                        size["wsm"], None))}
    for name, (written, read, call) in calls.items():
        for w in written:
            for r in (*written, *read):
                if r != w:
                    assert call({**place, w: place[r]}) == A, (name, w, r)
                    # the last 16 bytes of the other, and its first
                    assert call({**place, w: place[r] + (size[r] - 1) // 16 * 16}) == A, (name, w, r)
                    assert call({**place, r: place[w] + (size[w] - 1) // 16 * 16}) == A, (name, w, r)


@pytest.mark.parametrize("fmt", [5, 6])
def test_sizes_that_32_bits_do_not_count_are_refused(L, fmt):
    """A group of four rows has 4 scale_stride scales: 2^29 of them a row would pass 32 bits."""
    lib, V = L.lib(), ctypes.c_void_p
    K, N = 256, 8

    def desc(ss=8):
        return ctypes.byref(L.lbq_weights(fmt, 0, K, N, 1 << 24, 1 << 32, K // 2, ss))
    for ss in (2 ** 28 + 8, 2 ** 29, 2 ** 30, 2 ** 40):
        assert lib.lbq_workspace_bytes(desc(ss), 1) == 0
        assert lib.lbq_gemv(desc(ss), V(1 << 40), None, V(1 << 41), V(1 << 42), 1 << 30, None) == L.LBQ_ERR_SHAPE
        assert lib.lbq_expert_gemm(desc(ss), 2, V(1 << 40), 4, V(1 << 43), None, 1, 4, V(1 << 41), V(1 << 42), 1 << 30,
                                   None) == L.LBQ_ERR_SHAPE
    assert lib.lbq_workspace_bytes(desc(2 ** 28), 1) > 0
    for M in (2 ** 30 + 1, 2 ** 50, 2 ** 62):
        assert lib.lbq_workspace_bytes(desc(), M) == 0  # a bad argument
        assert lib.lbq_gemm(desc(), V(1 << 40), M, None, V(1 << 41), V(1 << 42), 1 << 62, None) == L.LBQ_ERR_SHAPE
    assert lib.lbq_workspace_bytes(desc(), 2 ** 30) > 2 * K * 2 ** 30


# ----------------------------------------------------------- weights that are not finite

@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [5, 6])
def test_a_nan_weight_packs_as_zero_and_alone(L, orc, fmt):
    """At each place of a word: the bytes of the same matrix with a zero there, and the
    oracle's; infinities saturate."""
    K, N = 256, 9
    W = synth.weights(N, K, 95)
    Z = W.clone()
    for i in range(8):
        W[i, 16 + i] = W[i, 200 + i] = float("nan")
        Z[i, 16 + i] = Z[i, 200 + i] = 0.0
    W[8], Z[8] = float("nan"), 0.0
    got, want = L.lbq_pack(fmt, W.cuda()), L.lbq_pack(fmt, Z.cuda())
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    W[3, 5], W[4, 6] = float("inf"), float("-inf")
    got = L.lbq_pack(fmt, W.cuda())
    codes, scales = orc.pack(fmt, W.numpy())
    assert np.array_equal(got.codes.cpu().numpy(), orc.group4(codes))
    assert np.array_equal(got.scales.cpu().numpy().view(np.uint16), orc.group4(scales))
    q, s = L.lbq_unpack(got)
    assert (q[3, 5], q[4, 6], s[3, 0], s[4, 0]) == (7, -8, 65504.0, 65504.0)


# --------------------------------------------------------------- rows recomputed in fp32

@pytest.mark.gpu
def test_rows_recomputed_for_longer_than_a_wait(L):
    """A whole tile of tokens that fp16 cannot hold, of more weights than are recomputed in
    the time that a wait lasts (5 to 8 ns a token and weight of a row, 6 s here).

    Sums: a thread adds K / 512 groups of 128 terms each, then four threads' sums: at most
    K / 512 + 128 + 3 additions one after another, each off by 2^-24 of S."""
    K, N, R = 3 << 20, 4, 256
    gen = torch.Generator("cuda").manual_seed(9)
    c = torch.randint(0, 256, (1, 1, 2 * K), dtype=torch.uint8, device="cuda", generator=gen)
    s = (torch.rand(1, 1, 4 * (K // 128), device="cuda", generator=gen) * 0.01 + 0.001).half().view(torch.int16)
    ew = L.ExpertWeights(6, K, N, 1, c, s)
    X = torch.randn(R, K, device="cuda", generator=gen, dtype=torch.bfloat16)
    X[:, 77] = 2.0 ** -60
    Y = L.lbq_expert_gemm(ew, X, torch.tensor([0, R], dtype=torch.int32, device="cuda"))
    assert L.lbq_device_fault() == 0
    W = _dense(L, L.PackedWeights(6, K, N, c[0], s[0]))
    for r in range(0, R, 16):
        x = X[r:r + 16].double()
        want, S = x @ W.t(), x.abs() @ W.abs().t()
        assert ((Y[r:r + 16].double() - want).abs() <= 2.0 ** -8 * want.abs() + (K / 512 + 131) * 2.0 ** -24 * S).all()


# ----------------------------------------- few rows and many: what is rounded, and where

def _few(M, N, K):
    """Whether lbq_gemm takes M rows on the path that rounds nothing before the output."""
    return M <= 8 or (M <= 32 and (M + 7) // 8 * N <= 2 ** 27 // K)


def _held(Y, X, W, f16, what):
    want, S = X.double() @ W.t(), X.double().abs() @ W.abs().t()
    err = (Y.double() - want).abs()
    lim = 2.0 ** -8 * want.abs() + (2.0 ** -12 + (2.0 ** -11 if f16 else 0.0)) * S
    assert (err <= lim).all(), f"{what}: {(err > lim).sum()} out of bound, worst {(err / lim).max()}"


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [5, 6])
@pytest.mark.parametrize("N,K,first", [(300, 1024, 33), (520, 5120, 33), (40000, 256, 33), (7168, 5120, 25),
                                       (10240, 5120, 17), (34816, 5120, 9)])
def test_dense_rows_on_both_sides_of_the_change(L, fmt, N, K, first):
    """The first number of rows that goes to the tensor cores, the one before, and others."""
    gen = torch.Generator("cuda").manual_seed(N)
    pw = L.lbq_pack(fmt, torch.randn(N, K, device="cuda", generator=gen) * 0.02)
    W = _dense(L, pw)
    X = torch.randn(64, K, device="cuda", generator=gen).to(torch.bfloat16)
    assert not _few(first, N, K) and _few(first - 1, N, K)
    for M in sorted({2, 4, 5, 8, 9, 16, 17, 24, 25, 32, 33, 64}):
        Y = L.lbq_gemm(pw, X[:M])
        _held(Y, X[:M], W, not _few(M, N, K), f"{M} rows")
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [5, 6])
@pytest.mark.parametrize("E,N,K", [(1, 70, 640), (6, 130, 1024), (40, 33, 384)])
def test_expert_rows_on_both_sides_of_the_change(L, fmt, E, N, K):
    """Up to eight slots an expert nothing is rounded before the output, however uneven."""
    gen = torch.Generator("cuda").manual_seed(E)
    ew = L.pack_experts(fmt, torch.randn(E, N, K, device="cuda", generator=gen) * 0.02)
    W = [_dense(L, L.PackedWeights(fmt, K, N, ew.codes[e], ew.scales[e])) for e in range(E)]
    X = torch.randn(8 * E + 1, K, device="cuda", generator=gen).to(torch.bfloat16)
    for R in (1, E, E + 1, 4 * E, 8 * E, 8 * E + 1):
        cuts = torch.randint(0, R + 1, (E - 1,), device="cuda", generator=gen).sort().values
        for inner in (cuts, torch.zeros_like(cuts), torch.full_like(cuts, R)):
            off = torch.cat([inner.new_zeros(1), inner, inner.new_full((1,), R)]).to(torch.int32)
            Y, o = L.lbq_expert_gemm(ew, X[:R], off), off.tolist()
            for e in range(E):
                if o[e] < o[e + 1]:
                    _held(Y[o[e]:o[e + 1]], X[o[e]:o[e + 1]], W[e], R > 8 * E, f"{R} rows, expert {e}")
    assert L.lbq_device_fault() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,K,lo,hi", [(5, 2048, 1024, 2048), (5, 2304, 1152, 2304), (6, 2048, 1024, 2048),
                                         (6, 3328, 1024, 3328), (5, 1536, 256, 1408)])
def test_a_range_of_k_of_a_wider_matrix(L, fmt, K, lo, hi):
    """Weights lo .. hi - 1 of every row, as a view; behind the last group's own bytes lies
    the output, which is neither read nor taken for a part of the matrix."""
    N, g = 10, {5: 32, 6: 128}[fmt]
    gen = torch.Generator("cuda").manual_seed(K)
    pw = L.lbq_pack(fmt, torch.randn(N, K, device="cuda", generator=gen) * 0.02)
    W = _dense(L, pw)[:, lo:hi]
    G, row = pw.codes.shape
    X = torch.randn(60, hi - lo, device="cuda", generator=gen).to(torch.bfloat16)
    end = (G - 1) * row + 2 * hi  # of the last group's bytes that belong to the range
    arena = torch.full((end + 2 * 60 * N,), 0xff, dtype=torch.uint8, device="cuda")
    arena[:end] = pw.codes.view(-1)[:end]
    codes = arena.as_strided((G, 2 * (hi - lo)), (row, 1), 2 * lo)
    scales = pw.scales[:, 4 * lo // g:]
    part = L.PackedWeights(fmt, hi - lo, N, codes, scales)
    for M in (1, 5, 60):
        Y = arena[end:end + 2 * M * N].view(torch.bfloat16).view(M, N)
        L.lbq_gemv(part, X[0], y=Y[0]) if M == 1 else L.lbq_gemm(part, X[:M], Y=Y)
        _held(Y, X[:M], W, M > 32, f"{M} rows")
    assert torch.equal(arena[:end], pw.codes.view(-1)[:end])
    assert L.lbq_device_fault() == 0
