"""The cases in which the 4-bit products and the expert operators are measured.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as a
user's program calls the library:

  product   4-bit weights with one fp16 scale per group of 32 or 128: y = W x for one
            token, for a list of independent products (a token's pass through a layer),
            and Y = X W^T for a batch of tokens
  route     token slots sorted by expert, the tokens' rows copied to the sorted order,
            and (grad) the gradient of that copy
  back      the experts' rows added up per token with the router's weights, and the
            gradients with respect to the rows and the weights
  experts   every sorted row times the 4-bit weights of its expert

A case names its operator in "op". Inputs come from the seed alone.
"""
import math

import torch

own = False

GROUP = {"q4g32": 32, "q4g128": 128}

# The four products of one decoder layer of the 27B shape: fused QKV, O, gate+up, down.
LAYER_27B = "5120x7168,5120x5120,5120x34816,17408x5120"


def listed():
    return [
        # The smallest product: latency of one call (the repository's tiny configuration).
        {"name": "product_tiny", "op": "product", "fmt": "q4g32", "M": 1, "shapes": "512x256"},
        # One token through one layer: the serving step, bound by the weights' bytes.
        {"name": "product_layer", "op": "product", "fmt": "q4g32", "M": 1, "shapes": LAYER_27B},
        # Five tokens (a speculative draft being verified) on the largest matrix.
        {"name": "product_m5", "op": "product", "fmt": "q4g128", "M": 5, "shapes": "5120x34816"},
        # A short prompt of odd length, rows of the output that fill no tile.
        {"name": "product_m333", "op": "product", "fmt": "q4g32", "M": 333, "shapes": "5120x7001"},
        # A long prompt: bound by the matrix instructions.
        {"name": "product_m4096", "op": "product", "fmt": "q4g128", "M": 4096, "shapes": "5120x34816"},
        # One token's routing: latency of the calls.
        {"name": "route_t1", "op": "route", "T": 1, "topk": 8, "E": 128, "K": 2048, "grad": False,
         "drop": 0.0},
        # A long prompt's routing with its gradient, some slots left out (experts that
        # another rank holds).
        {"name": "route_t4096", "op": "route", "T": 4096, "topk": 8, "E": 128, "K": 2048,
         "grad": True, "drop": 0.1},
        # A few tokens, an odd row width.
        {"name": "back_t7", "op": "back", "T": 7, "topk": 2, "E": 8, "N": 1001, "drop": 0.0},
        # A training batch.
        {"name": "back_t4096", "op": "back", "T": 4096, "topk": 8, "E": 128, "N": 2048,
         "drop": 0.1},
        # Three tokens being decoded: most experts untouched, one or two rows in the rest.
        {"name": "experts_t3", "op": "experts", "fmt": "q4g32", "T": 3, "topk": 8, "E": 128,
         "K": 2048, "N": 1536, "drop": 0.0},
        # A serving batch: every expert has a few rows.
        {"name": "experts_t64", "op": "experts", "fmt": "q4g128", "T": 64, "topk": 8, "E": 128,
         "K": 2048, "N": 1536, "drop": 0.0},
        # A long prompt: some 256 rows an expert, unevenly.
        {"name": "experts_t4096", "op": "experts", "fmt": "q4g32", "T": 4096, "topk": 8, "E": 128,
         "K": 2048, "N": 1536, "drop": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "list", "route", "back", "experts", "experts"])
    fmt = rng.choice(["q4g32", "q4g128"])
    if op in ("product", "list"):
        M = 1 if op == "list" else _log_int(rng, 1, 4096)
        shapes = []
        for _ in range(rng.randint(2, 8) if op == "list" else 1):
            K = 128 * _log_int(rng, 1, 136)
            shapes.append(f"{K}x{_log_int(rng, 64, 34816)}")
        return {"op": "product", "fmt": fmt, "M": M, "shapes": ",".join(shapes)}
    E = _log_int(rng, 4, 128)
    case = {"op": op, "E": E, "topk": rng.randint(1, min(8, E)), "T": _log_int(rng, 1, 4096),
            "drop": rng.choice([0.0, 0.0, 0.25])}
    if op == "route":
        return {**case, "K": _log_int(rng, 64, 4096), "grad": rng.random() < 0.5}
    if op == "back":
        return {**case, "N": _log_int(rng, 64, 4096)}
    return {**case, "fmt": fmt, "K": 128 * _log_int(rng, 1, 16), "N": _log_int(rng, 64, 1536)}


# ------------------------------------------------------------------------- inputs

def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _pack4(W, g):
    """fp32 W [N][K] -> (codes uint8 [ceil(N/4)][2K], scales int16 [ceil(N/4)][4 ss]): weights
    s (q - 8), s = max|w| / 7 in fp16, q the nearest of 0..15; rows in groups of four, weight
    8w + i of a row in bits 4 ((i >> 1) + 4 (i & 1)) of its 32-bit word w."""
    N, K = W.shape
    G, ng = (N + 3) // 4, K // g
    ss = (ng + 7) // 8 * 8
    blk = W.view(N, ng, g)
    s = (blk.abs().amax(-1) / 7.0).to(torch.float16)
    sf = s.float().unsqueeze(-1)
    q = torch.where(sf > 0, torch.round(blk / sf), torch.zeros_like(blk)).clamp_(-8, 7) + 8
    q = q.view(N, K // 8, 8).to(torch.int32)
    word = torch.zeros(4 * G, K // 8, dtype=torch.int32, device=W.device)
    for i in range(8):
        word[:N] |= q[:, :, i] << (4 * ((i >> 1) + 4 * (i & 1)))
    codes = word.view(G, 4, K // 8).transpose(1, 2).contiguous().view(torch.uint8).view(G, 2 * K)
    sp = torch.zeros(4 * G, ss, dtype=torch.float16, device=W.device)
    sp[:N, :ng] = s
    scales = sp.view(G, 4, ss).transpose(1, 2).contiguous().view(torch.int16).view(G, 4 * ss)
    return codes, scales


def _ids(T, topk, E, drop, gen, device):
    """Expert ids [T][topk]: the topk largest of a noisy router's logits that favours some
    experts, a share `drop` of the slots marked -1 (not computed here)."""
    logits = torch.randn(T, E, generator=gen, device=device)
    logits += 0.5 * torch.randn(1, E, generator=gen, device=device)
    w, ids = torch.softmax(logits, -1).topk(topk, -1)
    ids = ids.to(torch.int32)
    if drop > 0:
        ids[torch.rand(T, topk, generator=gen, device=device) < drop] = -1
    return ids, (w / w.sum(-1, keepdim=True)).contiguous()


def _sorted_places(ids, E):
    """(offsets [E+1], rows [T][topk], slots [T*topk]) of a stable sort by expert."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    count = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    count.index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = count[:E].cumsum(0).to(torch.int32)
    R = flat.numel()
    place = torch.empty_like(order)
    place[order] = torch.arange(R, device=ids.device)
    rows = torch.where(key < E, place, torch.full_like(place, -1)).to(torch.int32)
    behind = torch.arange(R, device=ids.device) >= offsets[E]
    slots = torch.where(behind, torch.full_like(order, -1), order).to(torch.int32)
    return offsets, rows.view_as(ids), slots


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * scale

    st = {"case": case}
    if case["op"] == "product":
        g = GROUP[case["fmt"]]
        st["w"], st["x"] = [], []
        for K, N in _shapes(case):
            st["w"].append((K, N, *_pack4(randn(N, K, scale=0.02), g)))
            st["x"].append(randn(case["M"], K).to(torch.bfloat16))
        if own:
            from bit_weight_only_ternary_b200 import lbq
            fmt = lbq.FORMATS[case["fmt"]]
            pw = [lbq.PackedWeights(fmt, K, N, c, s) for K, N, c, s in st["w"]]
            M = case["M"]
            st["y"] = [torch.empty((M, p.N), dtype=torch.bfloat16, device=dev) for p in pw]
            st["pw"] = pw
            if len(pw) > 1:
                st["list"] = lbq.ProductList([(p, x[0], None, y[0])
                                              for p, x, y in zip(pw, st["x"], st["y"])])
                st["ws"] = lbq.workspace_for_batch(st["list"])
            else:
                st["ws"] = lbq.workspace_for(pw[0], M)
        return st
    T, topk, E = case["T"], case["topk"], case["E"]
    R = T * topk
    st["ids"], st["weights"] = _ids(T, topk, E, case["drop"], gen, dev)
    if case["op"] == "route":
        st["x"] = randn(T, case["K"]).to(torch.bfloat16)
        st["xs"] = torch.zeros(R, case["K"], dtype=torch.bfloat16, device=dev)
        if case["grad"]:
            st["dxs"] = randn(R, case["K"]).to(torch.bfloat16)
        return st
    st["offsets"], st["rows"], st["slots"] = _sorted_places(st["ids"], E)
    if case["op"] == "back":
        st["y"] = randn(R, case["N"]).to(torch.bfloat16)
        st["dout"] = randn(T, case["N"]).to(torch.bfloat16)
        st["dy"] = torch.zeros(R, case["N"], dtype=torch.bfloat16, device=dev)
        return st
    g, K, N = GROUP[case["fmt"]], case["K"], case["N"]
    packed = [_pack4(randn(N, K, scale=0.02), g) for _ in range(E)]
    st["codes"] = torch.stack([p[0] for p in packed])
    st["scales"] = torch.stack([p[1] for p in packed])
    st["x"] = randn(T, K).to(torch.bfloat16)
    st["y"] = torch.zeros(R, N, dtype=torch.bfloat16, device=dev)
    if own:
        from bit_weight_only_ternary_b200 import lbq
        st["ew"] = lbq.ExpertWeights(lbq.FORMATS[case["fmt"]], K, N, E, st["codes"], st["scales"])
        st["ws"] = lbq.workspace_for_experts(st["ew"], R)
    return st


# --------------------------------------------------------------------- plain forms

def _unpack4(codes, scales, K, N, g):
    """fp32 weights [N][K] of one packed matrix."""
    G = codes.shape[0]
    word = codes.view(torch.int32).view(G, K // 8, 4).transpose(1, 2).reshape(4 * G, K // 8)
    q = torch.stack([(word >> (4 * ((i >> 1) + 4 * (i & 1)))) & 15 for i in range(8)], -1)
    q = q.view(4 * G, K)[:N].float() - 8.0
    s = scales.view(torch.float16).view(G, -1, 4).transpose(1, 2).reshape(4 * G, -1)
    return (q.view(N, K // g, g) * s[:N, :K // g].float().unsqueeze(-1)).view(N, K)


def _plain_product(st):
    g = GROUP[st["case"]["fmt"]]
    return [(x.float() @ _unpack4(c, s, K, N, g).t()).to(torch.bfloat16)
            for (K, N, c, s), x in zip(st["w"], st["x"])]


def _sum_slots(y, rows, weights):
    """out[t] = sum_j weights[t][j] y[rows[t][j]], slots of row -1 left out (fp32)."""
    out = torch.zeros(rows.shape[0], y.shape[1], device=y.device)
    for j in range(rows.shape[1]):
        keep = (rows[:, j] >= 0).float()
        w = keep if weights is None else keep * weights[:, j]
        out += w.unsqueeze(1) * y[rows[:, j].clamp(min=0).long()].float()
    return out


def _plain_route(st):
    c = st["case"]
    offsets, rows, slots = _sorted_places(st["ids"], c["E"])
    keep = slots >= 0
    token = (slots.clamp(min=0) // c["topk"]).long()
    st["xs"].copy_(torch.where(keep.unsqueeze(1), st["x"][token], st["xs"]))
    out = [offsets, rows, slots, st["xs"]]
    if c["grad"]:
        out.append(_sum_slots(st["dxs"], rows, None).to(torch.bfloat16))
    return out


def _plain_back(st):
    rows, w, y, dout = st["rows"], st["weights"], st["y"], st["dout"].float()
    out = _sum_slots(y, rows, w).to(torch.bfloat16)
    dw = torch.zeros_like(w)
    for j in range(rows.shape[1]):
        keep = rows[:, j] >= 0
        at = rows[:, j].clamp(min=0).long()
        dw[:, j] = torch.where(keep, (dout * y[at].float()).sum(-1), torch.zeros_like(w[:, j]))
        # slots that are left out write back what is there
        new = (w[:, j:j + 1] * dout).to(torch.bfloat16)
        st["dy"][at[keep]] = new[keep]
    return [out, st["dy"], dw]


def _plain_experts(st):
    c = st["case"]
    off = st["offsets"].tolist()
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            W = _unpack4(st["codes"][e], st["scales"][e], c["K"], c["N"], GROUP[c["fmt"]])
            x = st["x"][(st["slots"][lo:hi] // c["topk"]).long()].float()
            st["y"][lo:hi] = (x @ W.t()).to(torch.bfloat16)
    return st["y"]


# ---------------------------------------------------------------- the library's calls

def _own_run(st):
    from bit_weight_only_ternary_b200 import lbq
    c = st["case"]
    if c["op"] == "product":
        if len(st["pw"]) > 1:
            lbq.lbq_gemv_batch(st["list"], st["ws"])
        elif c["M"] == 1:
            lbq.lbq_gemv(st["pw"][0], st["x"][0][0], y=st["y"][0][0], workspace=st["ws"])
        else:
            lbq.lbq_gemm(st["pw"][0], st["x"][0], Y=st["y"][0], workspace=st["ws"])
        return st["y"]
    if c["op"] == "route":
        offsets, rows, slots = lbq.lbq_expert_sort(st["ids"], c["E"])
        lbq.lbq_expert_dispatch(st["x"], rows, out=st["xs"])
        out = [offsets, rows, slots, st["xs"]]
        if c["grad"]:
            out.append(lbq.lbq_expert_combine(st["dxs"], rows))
        return out
    if c["op"] == "back":
        out = lbq.lbq_expert_combine(st["y"], st["rows"], st["weights"])
        dy, dw = lbq.lbq_expert_combine_grad(st["dout"], st["y"], st["rows"], st["weights"],
                                             dY=st["dy"])
        return [out, dy, dw]
    return lbq.lbq_expert_gemm(st["ew"], st["x"], st["offsets"], slots=st["slots"],
                               topk=c["topk"], Y=st["y"], workspace=st["ws"])


def run(state):
    if own:
        return _own_run(state)
    return {"product": _plain_product, "route": _plain_route, "back": _plain_back,
            "experts": _plain_experts}[state["case"]["op"]](state)


# ----------------------------------------------------------------- what a pass needs

def _weight_bytes(K, N, g):
    return N * K // 2 + N * (K // g) * 2


def work(case):
    if case["op"] == "product":
        M, g = case["M"], GROUP[case["fmt"]]
        return {"bytes": sum(_weight_bytes(K, N, g) + 2 * M * (K + N) for K, N in _shapes(case)),
                "flops": sum(2 * M * K * N for K, N in _shapes(case))}
    T, topk, E = case["T"], case["topk"], case["E"]
    # the slots that are kept and the experts they touch, for one draw of the router
    ids, _ = _ids(T, topk, E, case["drop"], torch.Generator().manual_seed(0), "cpu")
    kept = int((ids >= 0).sum())
    touched = int(torch.unique(ids[ids >= 0]).numel())
    R = T * topk
    if case["op"] == "route":
        K = case["K"]
        n = 4 * (3 * R + E + 1) + 2 * T * K + 2 * kept * K
        if case["grad"]:
            n += 2 * kept * K + 2 * T * K
        return {"bytes": n, "flops": kept * K if case["grad"] else 0}
    if case["op"] == "back":
        N = case["N"]
        # rows and weights, y, dout read; out, dy, dw written (one reading of y serves both)
        return {"bytes": 4 * 3 * R + 2 * N * (2 * kept + 2 * T), "flops": 5 * kept * N}
    K, N = case["K"], case["N"]
    return {"bytes": touched * _weight_bytes(K, N, GROUP[case["fmt"]]) + 2 * T * K + 2 * kept * N
            + 4 * (kept + E + 1), "flops": 2 * kept * K * N}


# ------------------------------------------------------------- the definition, 64 bits

def _dense64(codes, scales, K, N, g):
    """fp64 weights [N][K], read byte by byte: byte b of a row's word holds nibbles 2b and
    2b + 1, and nibble p is weight 2 p (p < 4) or 2 (p - 4) + 1 of the word's eight."""
    G = codes.shape[0]
    b = codes.view(G, K // 8, 4, 4)  # group, word, row, byte
    nib = torch.stack([b & 15, b >> 4], -1).view(G, K // 8, 4, 8)
    place = [0, 4, 1, 5, 2, 6, 3, 7]  # the nibble that holds weight i
    q = nib[..., place].permute(0, 2, 1, 3).reshape(4 * G, K)[:N].double()
    s = scales.view(G, -1, 4).view(torch.float16).double().permute(0, 2, 1).reshape(4 * G, -1)
    return (q - 8.0) * s[:N, :K // g].repeat_interleave(g, 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "product":
        g = GROUP[case["fmt"]]
        return [torch.einsum("mk,nk->mn", x.double(), _dense64(c, s, K, N, g))
                for (K, N, c, s), x in zip(st["w"], st["x"])]
    T, topk, E = case["T"], case["topk"], case["E"]
    R, dev = T * topk, st["ids"].device
    # slots expert by expert, in slot order
    flat = st["ids"].cpu().view(-1).tolist()
    by = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            by[e].append(i)
    order = [i for b in by for i in b]
    offsets = [0]
    for b in by:
        offsets.append(offsets[-1] + len(b))
    kept = len(order)
    slot = torch.tensor(order, dtype=torch.long, device=dev)
    if case["op"] == "route":
        rows = torch.full((R,), -1, dtype=torch.int32, device=dev)
        rows[slot] = torch.arange(kept, dtype=torch.int32, device=dev)
        slots = torch.full((R,), -1, dtype=torch.int32, device=dev)
        slots[:kept] = slot.to(torch.int32)
        xs = st["xs"].double()
        xs[:kept] = st["x"].double()[slot // topk]
        out = [torch.tensor(offsets, dtype=torch.int32, device=dev), rows.view(T, topk), slots, xs]
        if case["grad"]:
            dx = torch.zeros(T, case["K"], dtype=torch.float64, device=dev)
            out.append(dx.index_add_(0, slot // topk, st["dxs"][:kept].double()))
        return out
    if case["op"] == "back":
        w = st["weights"].double().view(-1)[slot].unsqueeze(1)
        y, dout = st["y"].double(), st["dout"].double()
        out = torch.zeros(T, case["N"], dtype=torch.float64, device=dev)
        out.index_add_(0, slot // topk, w * y[:kept])
        dy = st["dy"].double()
        dy[:kept] = w * dout[slot // topk]
        dw = torch.zeros(R, dtype=torch.float64, device=dev)
        dw[slot] = (dout[slot // topk] * y[:kept]).sum(1)
        return [out, dy, dw.view(T, topk)]
    y = st["y"].double()
    for e in range(E):
        if by[e]:
            W = _dense64(st["codes"][e], st["scales"][e], case["K"], case["N"], GROUP[case["fmt"]])
            x = st["x"].double()[torch.tensor(by[e], device=dev) // topk]
            y[offsets[e]:offsets[e + 1]] = x @ W.t()
    return y
