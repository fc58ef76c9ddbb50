"""Work of the serving operators, for measurement: what a serving program calls
them on, their plain forms in torch, and their definitions in 64 bits.

Operators (include/moe_serve.h):

- quantize: bf16 -> E4M3 codes with one fp32 scale per block of 128. Rows
  (activations): blocks of 1 x 128; weights: blocks of 128 x 128.
    scale = amax(block) / 448,  code = E4M3(448 v / amax)  (0 and 0 for an all-zero block)
- gemm: the grouped product of block-scaled operands,
    out[p] = bf16(w[p] sum_b sa[p,b] sw[e,n/128,b] sum_{k in b} a[p,k] W[e,n,k])
  for the rows p of expert e; one expert is the dense product.
- experts: the expert stage for given routing: x quantised, gate/up with
  silu(g) u, its result quantised per 1 x 128, down, the weighted sum.
- few: the whole layer for at most 64 tokens: router, top-k, experts, sum,
  on bf16 weights or on E4M3 weights with 128 x 128 scales.

`own` selects the framework's calls; otherwise `run` is the plain form.
"""
import torch

own = False

FP8 = torch.float8_e4m3fn
E4M3_MAX = 448.0
BLOCK = 128


def listed():
    return [
        # A prefill batch's hidden states (the training batch of the Zipf workload: 16384 x 2048).
        {"name": "quantize_rows_16384x2048", "op": "quantize_rows", "rows": 16384, "K": 2048},
        # One projection of a 30B-A3B layer, at load time.
        {"name": "quantize_weights_128x768x2048", "op": "quantize_weights", "E": 128, "N": 768, "K": 2048},
        # One token through one dense projection (a shared expert): latency.
        {"name": "gemm_1x2048x2048", "op": "gemm", "M": 1, "E": 1, "N": 2048, "K": 2048, "weighted": False},
        # Ragged experts, a reduction and a width that end inside a block.
        {"name": "gemm_777x1000x720_e16", "op": "gemm", "M": 777, "E": 16, "N": 1000, "K": 720, "weighted": True},
        # The down projection of an 8192-token batch at the 30B-A3B shape.
        {"name": "gemm_65536x2048x768_e128", "op": "gemm", "M": 65536, "E": 128, "N": 2048, "K": 768, "weighted": True},
        # A dense product at the 235B-A22B hidden size.
        {"name": "gemm_8192x4096x4096", "op": "gemm", "M": 8192, "E": 1, "N": 4096, "K": 4096, "weighted": False},
        # A mixed decode batch just above the few-token layer: 12 rows per expert.
        {"name": "experts_t192", "op": "experts", "T": 192, "H": 2048, "E": 128, "k": 8, "I": 768, "zipf": 0.0},
        # A prefill of 4096 tokens with skewed routing (some experts empty, a few very long).
        {"name": "experts_t4096_zipf", "op": "experts", "T": 4096, "H": 2048, "E": 128, "k": 8, "I": 768, "zipf": 1.2},
        # Decoding one sequence, 30B-A3B.
        {"name": "few_bf16_t1", "op": "few", "fmt": "bf16", "T": 1, "H": 2048, "E": 128, "k": 8, "I": 768},
        # Decoding the largest few-token batch: nearly every expert is read.
        {"name": "few_bf16_t64", "op": "few", "fmt": "bf16", "T": 64, "H": 2048, "E": 128, "k": 8, "I": 768},
        # Decoding one sequence on 8-bit weights, 235B-A22B.
        {"name": "few_fp8_t1", "op": "few", "fmt": "fp8", "T": 1, "H": 4096, "E": 128, "k": 8, "I": 1536},
        # An odd decode batch on 8-bit weights, 30B-A3B.
        {"name": "few_fp8_t33", "op": "few", "fmt": "fp8", "T": 33, "H": 2048, "E": 128, "k": 8, "I": 768},
    ]


def draw(rng):
    def log(lo, hi):  # whole numbers spread over the logarithm
        return max(lo, min(hi, int(lo * (hi / lo) ** rng.random())))

    def times(n, lo, hi):  # multiples of n likewise
        return n * log(lo // n, hi // n)

    op = rng.choice(["quantize_rows", "quantize_weights", "gemm", "experts", "few", "few"])
    if op == "quantize_rows":
        return {"op": op, "rows": log(1, 16384), "K": times(8, 64, 2048)}
    if op == "quantize_weights":
        return {"op": op, "E": log(1, 128), "N": log(16, 768), "K": times(8, 64, 2048)}
    if op == "gemm":
        return {"op": op, "M": log(1, 8192), "E": log(1, 64), "N": times(8, 64, 2048), "K": times(16, 64, 2048),
                "weighted": rng.random() < 0.5}
    E = log(4, 128)
    k = rng.randint(1, min(8, E))
    H, I = times(64, 256, 2048), times(64, 64, 768)
    if op == "experts":
        return {"op": op, "T": log(1, 4096), "H": H, "E": E, "k": k, "I": I, "zipf": rng.choice([0.0, 1.2])}
    return {"op": op, "fmt": rng.choice(["bf16", "fp8"]), "T": log(1, 64), "H": H, "E": E, "k": k, "I": I}


def _blocks(n):
    return -(-n // BLOCK)


def _spread(v, dim, n):
    """One value per block of 128 along dim -> one per element."""
    return v.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


# ---- inputs -----------------------------------------------------------------


def _weights(g, E, N, K):
    return torch.randn(E, N, K, generator=g, device="cuda", dtype=torch.bfloat16) * 0.02


def _hidden(g, rows, K):
    """Hidden states: rows of different size, a few large channels."""
    size = torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    big = 1.0 + 7.0 * (torch.rand(1, K, generator=g, device="cuda") < 0.01)
    return (torch.randn(rows, K, generator=g, device="cuda") * size * big).bfloat16()


def _stored_weights(g, E, N, K):
    """Block-scaled weights as a checkpoint holds them: codes and scales."""
    q = torch.empty(E, N, K, device="cuda", dtype=FP8)
    s = torch.empty(E, _blocks(N), _blocks(K), device="cuda")
    step = max(1, (1 << 26) // (N * K))
    for e in range(0, E, step):
        w = _weights(g, min(step, E - e), N, K)
        q[e:e + step], s[e:e + step] = _quantize_weights(w)
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dev = case["op"], "cuda"
    i32, f32, u8, bf16 = torch.int32, torch.float32, torch.uint8, torch.bfloat16
    st = {"case": case}
    if op == "quantize_rows":
        rows, K = case["rows"], case["K"]
        st.update(x=_hidden(g, rows, K), q=torch.empty(rows, K, dtype=u8, device=dev),
                  scale=torch.empty(rows, _blocks(K), device=dev))
        return st
    if op == "quantize_weights":
        E, N, K = case["E"], case["N"], case["K"]
        st.update(w=_weights(g, E, N, K), q=torch.empty(E, N, K, dtype=u8, device=dev),
                  scale=torch.empty(E, _blocks(N), _blocks(K), device=dev))
        return st
    if op == "gemm":
        M, E, N, K = case["M"], case["E"], case["N"], case["K"]
        st["aq"], st["a_scale"] = _quantize_rows(_hidden(g, M, K))
        st["wq"], st["w_scale"] = _stored_weights(g, E, N, K)
        cuts = torch.randint(0, M + 1, (E - 1,), generator=g, device=dev).sort().values
        even = torch.arange(1, E, device=dev) * M // E
        ends = torch.zeros(E + 1, dtype=torch.int64, device=dev)
        ends[1:E] = (cuts + 3 * even) // 4  # ragged, around an even share
        ends[E] = M
        st["offsets"] = ends.to(i32)
        st["cap"] = int((ends[1:] - ends[:-1]).max())  # the plain form pads each expert's rows to the longest
        st["row_weight"] = torch.rand(M, generator=g, device=dev) if case["weighted"] else None
        st["out"] = torch.empty(M, N, dtype=bf16, device=dev)
        return st
    T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))
    if op == "experts" or case["fmt"] == "fp8":
        st["gate"], st["up"], st["down"] = (_stored_weights(g, E, I, H), _stored_weights(g, E, I, H),
                                            _stored_weights(g, E, H, I))
    else:
        st["gate"], st["up"], st["down"] = _weights(g, E, I, H), _weights(g, E, I, H), _weights(g, E, H, I)
    if op == "few":
        st.update(x=torch.randn(T, H, generator=g, device=dev).bfloat16(),
                  w_router=(0.02 * torch.randn(E, H, generator=g, device=dev)).bfloat16(),
                  bias=0.1 * torch.randn(E, generator=g, device=dev),
                  logits=torch.empty(T, E, device=dev), topk_idx=torch.empty(T, k, dtype=i32, device=dev),
                  topk_w=torch.empty(T, k, device=dev), y=torch.empty(T, H, dtype=bf16, device=dev),
                  ws=torch.empty(64 << 20, dtype=u8, device=dev))
        return st
    M = T * k
    rank = torch.randperm(E, generator=g, device=dev) + 1
    p = torch.softmax(torch.randn(T, E, generator=g, device=dev) - case["zipf"] * torch.log(rank.float()), 1)
    top, idx = torch.topk(p, k, dim=1)
    st.update(x=_hidden(g, T, H), topk_idx=idx.to(i32), topk_w=top / top.sum(1, keepdim=True),
              cap=int(torch.bincount(idx.reshape(-1), minlength=E).max()),
              counts=torch.empty(E, dtype=i32, device=dev), offsets=torch.empty(E + 1, dtype=i32, device=dev),
              sorted_to_flat=torch.empty(M, dtype=i32, device=dev), flat_to_sorted=torch.empty(M, dtype=i32, device=dev),
              row_token=torch.empty(M, dtype=i32, device=dev), row_weight=torch.empty(M, device=dev),
              xq=torch.empty(T, H, dtype=u8, device=dev), x_scale=torch.empty(T, _blocks(H), device=dev),
              aq=torch.empty(M, I, dtype=u8, device=dev), a_scale=torch.empty(M, _blocks(I), device=dev),
              o_perm=torch.empty(M, H, dtype=bf16, device=dev), y=torch.empty(T, H, dtype=bf16, device=dev),
              ws=torch.empty(1 << 30, dtype=u8, device=dev))
    return st


# ---- plain forms ------------------------------------------------------------


def _quantize_rows(x):
    """Blocks of 1 x 128. 448 v is exact for bf16 v, and one division follows."""
    R, K = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _blocks(K) * BLOCK - K)).view(R, _blocks(K), BLOCK)
    amax = v.abs().amax(2, keepdim=True)
    q = torch.where(amax > 0, v * E4M3_MAX / amax, torch.zeros_like(v)).to(FP8)
    return q.view(R, -1)[:, :K].contiguous(), amax[:, :, 0] / E4M3_MAX


def _quantize_weights(w):
    E, N, K = w.shape
    nb, kb = _blocks(N), _blocks(K)
    v = torch.nn.functional.pad(w.float(), (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(E, nb, BLOCK, kb, BLOCK)
    amax = v.abs().amax((2, 4), keepdim=True)
    q = torch.where(amax > 0, v * E4M3_MAX / amax, torch.zeros_like(v)).to(FP8)
    return q.view(E, nb * BLOCK, kb * BLOCK)[:, :N, :K].contiguous(), amax[:, :, 0, :, 0] / E4M3_MAX


def _dequantize_rows(q, s):
    return q.float() * _spread(s, 1, q.shape[1])


def _dequantize_weights(q, s):
    return q.float() * _spread(_spread(s, 1, q.shape[1]), 2, q.shape[2])


def _grouped(a, w, expert, pos, cap):
    """a [M,K] fp32 through its rows' experts' w [E,N,K], each expert's rows padded to cap."""
    padded = a.new_zeros(w.shape[0], cap, a.shape[1])
    padded[expert, pos] = a
    return torch.bmm(padded, w.transpose(1, 2))[expert, pos]


def _silu_mul(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def _plain_gemm(st):
    M = st["aq"].shape[0]
    row = torch.arange(M, device="cuda")
    off = st["offsets"].long()
    expert = torch.searchsorted(off[1:], row, right=True)
    out = _grouped(_dequantize_rows(st["aq"], st["a_scale"]), _dequantize_weights(st["wq"], st["w_scale"]), expert,
                   row - off[expert], st["cap"])
    if st["row_weight"] is not None:
        out = out * st["row_weight"][:, None]
    return out.bfloat16()


def _plain_experts(st):
    T, k = st["topk_idx"].shape
    E = st["gate"][0].shape[0]
    flat = st["topk_idx"].reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    expert = flat[order]
    counts = (flat[:, None] == torch.arange(E, device="cuda")).sum(0)
    pos = torch.arange(T * k, device="cuda") - (torch.cumsum(counts, 0) - counts)[expert]
    x = _dequantize_rows(*_quantize_rows(st["x"]))[order // k]
    g = _grouped(x, _dequantize_weights(*st["gate"]), expert, pos, st["cap"])
    u = _grouped(x, _dequantize_weights(*st["up"]), expert, pos, st["cap"])
    a = _dequantize_rows(*_quantize_rows(_silu_mul(g, u)))
    o = _grouped(a, _dequantize_weights(*st["down"]), expert, pos, st["cap"])
    by_slot = torch.empty_like(o)
    by_slot[order] = o
    return (by_slot.view(T, k, -1) * st["topk_w"][:, :, None]).sum(1).bfloat16()


def _plain_few(st):
    """The k experts of each token, gathered. Logits in 64 bits, rounded once:
    a logit next to the k-th one decides which expert is read."""
    case, x = st["case"], st["x"].float()
    T, k = case["T"], case["k"]
    logits = (st["x"].double() @ st["w_router"].double().T + st["bias"].double()).float()
    idx = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]  # ties: the lower index first
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    top = p.gather(1, idx)
    w = top / (top.sum(1, keepdim=True) + 1e-20)
    pair, tok = idx.reshape(-1), torch.arange(T, device="cuda").repeat_interleave(k)
    if case["fmt"] == "fp8":
        gate, up, down = (_dequantize_weights(q[pair], s[pair]) for q, s in (st["gate"], st["up"], st["down"]))
    else:
        gate, up, down = (m[pair].float() for m in (st["gate"], st["up"], st["down"]))
    a = _silu_mul(torch.bmm(gate, x[tok][:, :, None]), torch.bmm(up, x[tok][:, :, None]))
    o = torch.bmm(down, a).view(T, k, -1)
    return {"logits": logits, "idx": idx.to(torch.int32), "w": w, "y": (o * w[:, :, None]).sum(1).bfloat16()}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _own(state)
    if op == "quantize_rows":
        q, s = _quantize_rows(state["x"])
        return {"q": q, "scale": s}
    if op == "quantize_weights":
        q, s = _quantize_weights(state["w"])
        return {"q": q, "scale": s}
    if op == "gemm":
        return _plain_gemm(state)
    if op == "experts":
        return _plain_experts(state)
    return _plain_few(state)


# ---- the framework's calls --------------------------------------------------


def _own(st):
    from mixture_experts_expert_amd import binding as B

    case = st["case"]
    op = case["op"]
    if op == "quantize_rows":
        B.moe_quantize_fp8_block_rows(case["rows"], case["K"], st["x"], st["q"], st["scale"])
        return {"q": st["q"].view(FP8), "scale": st["scale"]}
    if op == "quantize_weights":
        B.moe_quantize_fp8_block_weights(case["E"], case["N"], case["K"], st["w"], st["q"], st["scale"])
        return {"q": st["q"].view(FP8), "scale": st["scale"]}
    if op == "gemm":
        B.moe_gemm_fp8_block(case["M"], case["E"], case["N"], case["K"], st["aq"], st["a_scale"], st["offsets"], st["wq"],
                             st["w_scale"], st["row_weight"], st["out"])
        return st["out"]
    s = B.shape(case["T"], case["H"], case["E"], case["k"], case["I"], torch.bfloat16)
    if op == "experts":
        B.moe_experts_fp8_block(s, st["x"], st["topk_idx"], st["topk_w"], *st["gate"], *st["up"], *st["down"],
                                st["counts"], st["offsets"], st["sorted_to_flat"], st["flat_to_sorted"],
                                st["row_token"], st["row_weight"], st["xq"], st["x_scale"], st["aq"], st["a_scale"],
                                st["o_perm"], st["y"], st["ws"])
        return st["y"]
    out = (st["logits"], st["topk_idx"], st["topk_w"], st["y"], st["ws"])
    if case["fmt"] == "fp8":
        B.moe_forward_few_fp8_block(s, st["x"], st["w_router"], st["bias"], *st["gate"], *st["up"], *st["down"], *out)
    else:
        B.moe_forward_few(s, st["x"], st["w_router"], st["bias"], st["gate"], st["up"], st["down"], *out)
    return {"logits": st["logits"], "idx": st["topk_idx"], "w": st["topk_w"], "y": st["y"]}


# ---- what a pass cannot do without ------------------------------------------


def work(case):
    op = case["op"]
    if op == "quantize_rows":
        n = case["rows"] * case["K"]
        return {"bytes": 3 * n + 4 * case["rows"] * _blocks(case["K"]), "flops": 3 * n}
    if op == "quantize_weights":
        n = case["E"] * case["N"] * case["K"]
        return {"bytes": 3 * n + 4 * case["E"] * _blocks(case["N"]) * _blocks(case["K"]), "flops": 3 * n}
    if op == "gemm":
        M, E, N, K = (case[n] for n in ("M", "E", "N", "K"))
        return {"bytes": M * K + 4 * M * _blocks(K) + min(E, M) * (N * K + 4 * _blocks(N) * _blocks(K)) + 2 * M * N,
                "flops": 2 * M * N * K}
    T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))
    if op == "experts":  # the experts that a batch reaches: all but a few
        return {"bytes": 4 * T * H + 8 * T * k + min(E, T * k) * 3 * H * I, "flops": 6 * T * k * H * I}
    reached = E * (1.0 - (1.0 - k / E) ** T)  # distinct experts of T tokens, each k of E
    each = 2 if case["fmt"] == "bf16" else 1
    return {"bytes": 4 * T * H + 2 * E * H + 4 * T * (E + 2 * k) + reached * 3 * H * I * each,
            "flops": 6 * T * k * H * I + 2 * T * E * H}


# ---- the definitions in 64 bits ---------------------------------------------


def _e4m3_64(v):
    """The E4M3 value nearest to v (float64, |v| <= 448), ties to the even code."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step  # torch rounds halves to even


def _block_quantized_64(v, rows):
    """(values v / scale, scales) of a float64 matrix with blocks of rows x 128."""
    R, K = v.shape
    scales = torch.zeros(-(-R // rows), _blocks(K), dtype=torch.float64, device=v.device)
    q = torch.zeros_like(v)
    for b in range(_blocks(K)):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        amax = part.abs().amax(1)
        if rows > 1:
            for n in range(scales.shape[0]):
                amax[n * rows:(n + 1) * rows] = amax[n * rows:(n + 1) * rows].amax()
        scales[:, b] = amax[::rows] / E4M3_MAX
        safe = torch.where(amax > 0, amax, torch.ones_like(amax))[:, None]
        q[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3_64(part * E4M3_MAX / safe)
    return q, scales


def _deq_64(q, s, rows):
    out = q.double().clone()
    for n in range(s.shape[0]):
        for b in range(s.shape[1]):
            out[n * rows:(n + 1) * rows, b * BLOCK:(b + 1) * BLOCK] *= s[n, b].double()
    return out


def _deq_rows_64(q, s):
    out = q.double().clone()
    for b in range(s.shape[1]):
        out[:, b * BLOCK:(b + 1) * BLOCK] *= s[:, b:b + 1].double()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize_rows":
        q, s = _block_quantized_64(st["x"].double(), 1)
        return {"q": q, "scale": s}
    if op == "quantize_weights":
        qs, ss = zip(*(_block_quantized_64(w.double(), BLOCK) for w in st["w"]))
        return {"q": torch.stack(qs), "scale": torch.stack(ss)}
    if op == "gemm":
        a = _deq_rows_64(st["aq"], st["a_scale"])
        out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        ends = st["offsets"].tolist()
        for e in range(case["E"]):
            if ends[e + 1] > ends[e]:
                w = _deq_64(st["wq"][e], st["w_scale"][e], BLOCK)
                out[ends[e]:ends[e + 1]] = a[ends[e]:ends[e + 1]] @ w.T
        return out if st["row_weight"] is None else out * st["row_weight"].double()[:, None]
    T, E, k = case["T"], case["E"], case["k"]
    quantised = op == "experts" or case["fmt"] == "fp8"

    def matrix(m, e):
        return _deq_64(m[0][e], m[1][e], BLOCK) if quantised else m[e].double()

    logits = None
    if op == "few":
        x = st["x"].double()
        logits = x @ st["w_router"].double().T + st["bias"].double()
        idx = torch.argsort(logits.float(), dim=1, descending=True, stable=True)[:, :k]
        p = torch.softmax(logits, 1).gather(1, idx)
        w = p / (p.sum(1, keepdim=True) + 1e-20)
    else:
        q, s = _block_quantized_64(st["x"].double(), 1)
        x = _deq_rows_64(q, s)
        idx, w = st["topk_idx"].long(), st["topk_w"].double()
    y = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
    for e in range(E):
        tok, slot = torch.nonzero(idx == e, as_tuple=True)
        if tok.numel() == 0:
            continue
        g, u = x[tok] @ matrix(st["gate"], e).T, x[tok] @ matrix(st["up"], e).T
        a = g * torch.sigmoid(g) * u
        if op == "experts":
            a = _deq_rows_64(*_block_quantized_64(a, 1))
        y.index_add_(0, tok, (a @ matrix(st["down"], e).T) * w[tok, slot][:, None])
    if op == "experts":
        return y
    return {"logits": logits, "idx": idx.to(torch.int32), "w": w, "y": y}
