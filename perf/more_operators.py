"""Work of the 8-bit integer operators, for measurement: what serving and training
programs call them on, their plain forms in torch, and their definitions in 64 bits.

Operators (include/moe_serve.h, include/moe.h). Codes are whole numbers in
[-127, 127], scale = amax / 127, code = the whole number nearest to 127 v / amax
(halves to even; 0 and 0 where amax is 0):

- quantize_rows: bf16 -> codes with one fp32 scale per row (a token, or an
  output channel of a weight).
- save_rows: hidden states kept for the backward pass in 8 bits, one fp32 scale
  per 64 of a row, and read back: bf16(code scale).
- gemm: the grouped product of such operands,
    out[p,n] = bf16(w[p] sa[p] sw[e,n] sum_k a[p,k] W[e,n,k])
  for the rows p of expert e; one expert is the dense product.
- experts: the expert stage for given routing: x quantised per token, gate/up
  with silu(g) u, its result quantised per row, down, the weighted sum.
- few: the whole layer for at most 64 tokens on 8-bit weights: router, top-k,
  experts, sum.
- saved_forward: gate/up of the training step that keeps g and u in 8 bits (one
  scale per 64 of a row): a = bf16(silu(g) u) from the exact g and u, and the
  kept ones read back.
- saved_backward: the down projection's data gradient from the kept g and u,
    dA = dy[t] W_down,  a = silu(g) u,  s = sigmoid(g),
    dG = w dA u s (1 + g (1 - s)),  dU = w dA silu(g),  a_w = w a,
    d_topk_w[t,j] = <dA, a>
  for sorted row p of token t and slot j with routing weight w.

`own` selects the framework's calls; otherwise `run` is the plain form.
"""
import torch

own = False

SAVED = 64  # columns per scale of kept activations


def listed():
    return [
        # A prefill batch's hidden states (the Zipf workload's 16384 tokens), one scale per token.
        {"name": "quantize_rows_16384x2048", "op": "quantize_rows", "rows": 16384, "K": 2048},
        # A training batch's hidden states, kept for the backward pass and read back there.
        {"name": "save_rows_8192x2048", "op": "save_rows", "rows": 8192, "K": 2048},
        # One token through one dense projection (a shared expert): latency.
        {"name": "gemm_1x2048x2048", "op": "gemm", "M": 1, "E": 1, "N": 2048, "K": 2048, "weighted": False},
        # The down projection of an 8192-token batch at the 30B-A3B shape.
        {"name": "gemm_65536x2048x768_e128", "op": "gemm", "M": 65536, "E": 128, "N": 2048, "K": 768, "weighted": True},
        # A mixed decode batch just above the few-token layer: 12 rows per expert.
        {"name": "experts_t192", "op": "experts", "T": 192, "H": 2048, "E": 128, "k": 8, "I": 768, "zipf": 0.0},
        # A prefill of 4096 tokens with skewed routing (some experts empty, a few very long).
        {"name": "experts_t4096_zipf", "op": "experts", "T": 4096, "H": 2048, "E": 128, "k": 8, "I": 768, "zipf": 1.2},
        # Decoding one sequence, 235B-A22B.
        {"name": "few_t1", "op": "few", "T": 1, "H": 4096, "E": 128, "k": 8, "I": 1536},
        # An odd decode batch, 30B-A3B.
        {"name": "few_t33", "op": "few", "T": 33, "H": 2048, "E": 128, "k": 8, "I": 768},
        # Training steps: a ragged small layer with skewed routing, and the 30B-A3B layer's batch.
        {"name": "saved_forward_t500_zipf", "op": "saved_forward", "T": 500, "H": 512, "E": 16, "k": 4, "I": 320,
         "zipf": 1.2},
        {"name": "saved_forward_t8192", "op": "saved_forward", "T": 8192, "H": 2048, "E": 128, "k": 8, "I": 768,
         "zipf": 0.0},
        {"name": "saved_backward_t500_zipf", "op": "saved_backward", "T": 500, "H": 512, "E": 16, "k": 4, "I": 320,
         "zipf": 1.2},
        {"name": "saved_backward_t8192", "op": "saved_backward", "T": 8192, "H": 2048, "E": 128, "k": 8, "I": 768,
         "zipf": 0.0},
    ]


def draw(rng):
    def log(lo, hi):  # whole numbers spread over the logarithm
        return max(lo, min(hi, int(lo * (hi / lo) ** rng.random())))

    def times(n, lo, hi):  # multiples of n likewise
        return n * log(lo // n, hi // n)

    op = rng.choice(["quantize_rows", "save_rows", "gemm", "gemm", "experts", "few", "saved_forward", "saved_backward"])
    if op in ("quantize_rows", "save_rows"):
        return {"op": op, "rows": log(1, 16384 if op == "quantize_rows" else 8192), "K": times(8, 64, 2048)}
    if op == "gemm":
        return {"op": op, "M": log(1, 8192), "E": log(1, 64), "N": times(8, 64, 2048), "K": times(16, 64, 2048),
                "weighted": rng.random() < 0.5}
    E = log(4, 128)
    k = rng.randint(1, min(8, E))
    case = {"op": op, "T": log(1, {"few": 64, "experts": 4096}.get(op, 8192)), "H": times(64, 256, 2048), "E": E, "k": k,
            "I": times(64, 64, 768)}
    if op != "few":
        case["zipf"] = rng.choice([0.0, 1.2]) if case["T"] <= 4096 else 0.0
    return case


# ---- inputs -----------------------------------------------------------------


def _weights(g, E, N, K):
    return torch.randn(E, N, K, generator=g, device="cuda", dtype=torch.bfloat16) * 0.02


def _hidden(g, rows, K):
    """Hidden states: rows of different size, a few large channels."""
    size = torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    big = 1.0 + 7.0 * (torch.rand(1, K, generator=g, device="cuda") < 0.01)
    return (torch.randn(rows, K, generator=g, device="cuda") * size * big).bfloat16()


def _stored_weights(g, E, N, K):
    """8-bit weights as a checkpoint holds them: codes, and a scale per output channel."""
    q = torch.empty(E, N, K, device="cuda", dtype=torch.int8)
    s = torch.empty(E, N, device="cuda")
    step = max(1, (1 << 26) // (N * K))
    for e in range(0, E, step):
        w = _weights(g, min(step, E - e), N, K)
        q[e:e + step], s[e:e + step] = _quantize(w.float())
    return q, s


def _routing(g, st, T, E, k, zipf):
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    p = torch.softmax(torch.randn(T, E, generator=g, device="cuda") - zipf * torch.log(rank.float()), 1)
    top, idx = torch.topk(p, k, dim=1)
    st.update(topk_idx=idx.to(torch.int32), topk_w=top / top.sum(1, keepdim=True),
              cap=int(torch.bincount(idx.reshape(-1), minlength=E).max()))  # the plain form pads each expert's rows to it


def _sorted(st, E):
    """What the sort gives the products: each expert's rows, their tokens, weights and slots."""
    flat = st["topk_idx"].reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    k = st["topk_idx"].shape[1]
    ends = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    ends[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    st.update(offsets=ends.to(torch.int32), sorted_to_flat=order.to(torch.int32), row_token=(order // k).to(torch.int32),
              row_weight=st["topk_w"].reshape(-1)[order].contiguous())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dev = case["op"], "cuda"
    i8, i32, f32, u8, bf16 = torch.int8, torch.int32, torch.float32, torch.uint8, torch.bfloat16
    st = {"case": case}

    def buf(*size, dtype=f32):
        return torch.empty(*size, dtype=dtype, device=dev)

    if op in ("quantize_rows", "save_rows"):
        rows, K = case["rows"], case["K"]
        st.update(x=_hidden(g, rows, K), q=buf(rows, K, dtype=i8))
        if op == "quantize_rows":
            st["scale"] = buf(rows)
        else:
            st.update(scale=buf(rows, -(-K // SAVED)), back=buf(rows, K, dtype=bf16))
        return st
    if op == "gemm":
        M, E, N, K = case["M"], case["E"], case["N"], case["K"]
        st["aq"], st["a_scale"] = _quantize(_hidden(g, M, K).float())
        st["wq"], st["w_scale"] = _stored_weights(g, E, N, K)
        cuts = torch.randint(0, M + 1, (E - 1,), generator=g, device=dev).sort().values
        even = torch.arange(1, E, device=dev) * M // E
        ends = torch.zeros(E + 1, dtype=torch.int64, device=dev)
        ends[1:E] = (cuts + 3 * even) // 4  # ragged, around an even share
        ends[E] = M
        st["offsets"] = ends.to(i32)
        st["cap"] = int((ends[1:] - ends[:-1]).max())
        st["row_weight"] = torch.rand(M, generator=g, device=dev) if case["weighted"] else None
        st["out"] = buf(M, N, dtype=bf16)
        return st
    T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))
    M = T * k
    if op == "few":
        st.update(gate=_stored_weights(g, E, I, H), up=_stored_weights(g, E, I, H), down=_stored_weights(g, E, H, I),
                  x=torch.randn(T, H, generator=g, device=dev).bfloat16(),
                  w_router=(0.02 * torch.randn(E, H, generator=g, device=dev)).bfloat16(),
                  bias=0.1 * torch.randn(E, generator=g, device=dev),
                  logits=buf(T, E), topk_idx=buf(T, k, dtype=i32), topk_w=buf(T, k), y=buf(T, H, dtype=bf16),
                  ws=buf(64 << 20, dtype=u8))
        return st
    _routing(g, st, T, E, k, case["zipf"])
    if op == "experts":
        st.update(gate=_stored_weights(g, E, I, H), up=_stored_weights(g, E, I, H), down=_stored_weights(g, E, H, I),
                  x=_hidden(g, T, H), counts=buf(E, dtype=i32), offsets=buf(E + 1, dtype=i32),
                  sorted_to_flat=buf(M, dtype=i32), flat_to_sorted=buf(M, dtype=i32), row_token=buf(M, dtype=i32),
                  row_weight=buf(M), xq=buf(T, H, dtype=i8), x_scale=buf(T), aq=buf(M, I, dtype=i8), a_scale=buf(M),
                  o_perm=buf(M, H, dtype=bf16), y=buf(T, H, dtype=bf16), ws=buf((64 << 20) + 4 * M * I, dtype=u8))
        return st
    _sorted(st, E)
    blocks = -(-I // SAVED)
    if op == "saved_forward":
        st.update(x=torch.randn(T, H, generator=g, device=dev).bfloat16(), w_gate=_weights(g, E, I, H),
                  w_up=_weights(g, E, I, H), gq=buf(M, I, dtype=i8), g_scale=buf(M, blocks), uq=buf(M, I, dtype=i8),
                  u_scale=buf(M, blocks), a=buf(M, I, dtype=bf16), g=buf(M, I, dtype=bf16), u=buf(M, I, dtype=bf16))
        return st
    st["gq"], st["g_scale"] = _save(0.9 * torch.randn(M, I, generator=g, device=dev))
    st["uq"], st["u_scale"] = _save(0.9 * torch.randn(M, I, generator=g, device=dev))
    st.update(dy=torch.randn(T, H, generator=g, device=dev).bfloat16(), w_down=_weights(g, E, H, I),
              dgu=buf(M, 2 * I, dtype=bf16), a_w=buf(M, I, dtype=bf16), d_topk_w=buf(T, k), ws=buf(64 << 20, dtype=u8))
    return st


# ---- plain forms ------------------------------------------------------------


def _quantize(v):
    """fp32 [.., K], one scale per row. 127 v is exact for bf16 v, and one division follows."""
    amax = v.abs().amax(-1, keepdim=True)
    q = torch.where(amax > 0, torch.round(v * 127.0 / amax), torch.zeros_like(v)).to(torch.int8)
    return q, amax[..., 0] / 127.0


def _save(v):
    """fp32 [rows, K], one scale per 64 of a row."""
    rows, K = v.shape
    n = -(-K // SAVED)
    q, s = _quantize(torch.nn.functional.pad(v, (0, n * SAVED - K)).view(rows, n, SAVED))
    return q.view(rows, -1)[:, :K].contiguous(), s


def _restore(q, s):
    return q.float() * s.repeat_interleave(SAVED, 1)[:, :q.shape[1]]


def _grouped(a, w, expert, pos, cap):
    """a [M,K] fp32 through its rows' experts' w [E,N,K], each expert's rows padded to cap."""
    padded = a.new_zeros(w.shape[0], cap, a.shape[1])
    padded[expert, pos] = a
    return torch.bmm(padded, w.transpose(1, 2))[expert, pos]


def _rows_of(offsets, M):
    """(expert, place among its rows) of each sorted row."""
    row = torch.arange(M, device="cuda")
    off = offsets.long()
    expert = torch.searchsorted(off[1:], row, right=True)
    return expert, row - off[expert]


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _plain_gemm(st):
    expert, pos = _rows_of(st["offsets"], st["aq"].shape[0])
    sums = _grouped(st["aq"].float(), st["wq"].float(), expert, pos, st["cap"])
    out = sums * st["a_scale"][:, None] * st["w_scale"][expert]
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

    def product(q, s, w):  # codes q with row scales s through the stacked weight w
        return _grouped(q.float(), w[0].float(), expert, pos, st["cap"]) * s[:, None] * w[1][expert]

    xq, xs = _quantize(st["x"].float())
    token = order // k
    g, u = product(xq[token], xs[token], st["gate"]), product(xq[token], xs[token], st["up"])
    o = product(*_quantize(_silu(g) * u), st["down"])
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

    def product(m, v):
        return torch.bmm(m[0][pair].float(), v[:, :, None])[:, :, 0] * m[1][pair]

    a = _silu(product(st["gate"], x[tok])) * product(st["up"], x[tok])
    o = product(st["down"], a).view(T, k, -1)
    return {"logits": logits, "idx": idx.to(torch.int32), "w": w, "y": (o * w[:, :, None]).sum(1).bfloat16()}


def _plain_saved_forward(st):
    x = st["x"].float()[st["row_token"].long()]
    expert, pos = _rows_of(st["offsets"], x.shape[0])
    g = _grouped(x, st["w_gate"].float(), expert, pos, st["cap"])
    u = _grouped(x, st["w_up"].float(), expert, pos, st["cap"])
    return {"a": (_silu(g) * u).bfloat16(), "g": _restore(*_save(g)).bfloat16(), "u": _restore(*_save(u)).bfloat16()}


def _plain_saved_backward(st):
    dy = st["dy"].float()[st["row_token"].long()]
    expert, pos = _rows_of(st["offsets"], dy.shape[0])
    dA = _grouped(dy, st["w_down"].float().transpose(1, 2), expert, pos, st["cap"])
    g, u, w = _restore(st["gq"], st["g_scale"]), _restore(st["uq"], st["u_scale"]), st["row_weight"][:, None]
    s = 1.0 / (1.0 + torch.exp(-g))
    a = g * s * u
    d_topk_w = torch.empty_like(st["topk_w"])
    d_topk_w.view(-1)[st["sorted_to_flat"].long()] = (dA * a).sum(1)
    dgu = torch.cat([w * dA * u * s * (1.0 + g * (1.0 - s)), w * dA * g * s], 1)
    return {"dgu": dgu.bfloat16(), "a_w": (w * a).bfloat16(), "d_topk_w": d_topk_w}


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    if op == "quantize_rows":
        q, s = _quantize(state["x"].float())
        return {"q": q, "scale": s}
    if op == "save_rows":
        q, s = _save(state["x"].float())
        return {"q": q, "scale": s, "back": _restore(q, s).bfloat16()}
    return {"gemm": _plain_gemm, "experts": _plain_experts, "few": _plain_few, "saved_forward": _plain_saved_forward,
            "saved_backward": _plain_saved_backward}[op](state)


# ---- the framework's calls --------------------------------------------------


def _own(st):
    from mixture_experts_expert_amd import binding as B

    case = st["case"]
    op = case["op"]
    if op == "quantize_rows":
        B.moe_quantize_i8_rows(case["rows"], case["K"], st["x"], st["q"], st["scale"])
        return {"q": st["q"], "scale": st["scale"]}
    if op == "save_rows":
        B.moe_quantize_ckpt8(case["rows"], case["K"], st["x"], st["q"], st["scale"])
        B.moe_dequantize_ckpt8(case["rows"], case["K"], st["q"], st["scale"], st["back"])
        return {"q": st["q"], "scale": st["scale"], "back": st["back"]}
    if op == "gemm":
        B.moe_gemm_i8(case["M"], case["E"], case["N"], case["K"], st["aq"], st["a_scale"], st["offsets"], st["wq"],
                      st["w_scale"], st["row_weight"], st["out"])
        return st["out"]
    s = B.shape(case["T"], case["H"], case["E"], case["k"], case["I"], torch.bfloat16)
    if op == "experts":
        B.moe_experts_i8(s, st["x"], st["topk_idx"], st["topk_w"], *st["gate"], *st["up"], *st["down"], st["counts"],
                         st["offsets"], st["sorted_to_flat"], st["flat_to_sorted"], st["row_token"], st["row_weight"],
                         st["xq"], st["x_scale"], st["aq"], st["a_scale"], st["o_perm"], st["y"], st["ws"])
        return st["y"]
    if op == "few":
        B.moe_forward_few_i8(s, st["x"], st["w_router"], st["bias"], *st["gate"], *st["up"], *st["down"], st["logits"],
                             st["topk_idx"], st["topk_w"], st["y"], st["ws"])
        return {"logits": st["logits"], "idx": st["topk_idx"], "w": st["topk_w"], "y": st["y"]}
    saved = (st["gq"], st["g_scale"], st["uq"], st["u_scale"])
    if op == "saved_forward":
        M, I = st["a"].shape
        B.moe_gemm_gate_up_ckpt8(s, st["x"], st["row_token"], st["offsets"], st["w_gate"], st["w_up"], *saved, st["a"])
        B.moe_dequantize_ckpt8(M, I, st["gq"], st["g_scale"], st["g"])
        B.moe_dequantize_ckpt8(M, I, st["uq"], st["u_scale"], st["u"])
        return {"a": st["a"], "g": st["g"], "u": st["u"]}
    B.moe_gemm_down_dgrad_ckpt8(s, st["dy"], st["row_token"], st["row_weight"], st["sorted_to_flat"], st["offsets"],
                                st["w_down"], *saved, st["dgu"], st["a_w"], st["d_topk_w"], st["ws"])
    return {"dgu": st["dgu"], "a_w": st["a_w"], "d_topk_w": st["d_topk_w"]}


# ---- what a pass cannot do without ------------------------------------------


def work(case):
    op = case["op"]
    if op == "quantize_rows":
        n = case["rows"] * case["K"]
        return {"bytes": 3 * n + 4 * case["rows"], "flops": 3 * n}
    if op == "save_rows":  # x read, codes, scales and the restored x written
        n = case["rows"] * case["K"]
        return {"bytes": 5 * n + 4 * case["rows"] * -(-case["K"] // SAVED), "flops": 4 * n}
    if op == "gemm":
        M, E, N, K = (case[n] for n in ("M", "E", "N", "K"))
        e = min(E, M)
        return {"bytes": M * K + 4 * M + e * N * (K + 4) + 2 * M * N, "flops": 2 * M * N * K}
    T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))
    M = T * k
    if op == "experts":  # the experts that a batch reaches: all but a few
        return {"bytes": 4 * T * H + 8 * M + min(E, M) * (3 * H * I + 8 * I + 4 * H), "flops": 6 * M * H * I}
    if op == "few":  # distinct experts of T tokens, each k of E
        reached = E * (1.0 - (1.0 - k / E) ** T)
        return {"bytes": 4 * T * H + 2 * E * H + 4 * T * (E + 2 * k) + reached * (3 * H * I + 8 * I + 4 * H),
                "flops": 6 * M * H * I + 2 * T * E * H}
    kept = 2 * M * (I + 4 * -(-I // SAVED))  # codes and scales of g and u
    if op == "saved_forward":  # a, and the restored g and u
        return {"bytes": 2 * T * H + min(E, M) * 4 * I * H + kept + 6 * M * I, "flops": 4 * M * I * H}
    return {"bytes": 2 * T * H + min(E, M) * 2 * I * H + kept + 6 * M * I + 12 * M, "flops": 2 * M * I * H}


# ---- the definitions in 64 bits ---------------------------------------------


def _codes_64(v, width):
    """(codes, scales) of a float64 matrix with one scale per `width` columns, block by block."""
    q = torch.zeros_like(v)
    scales = []
    for at in range(0, v.shape[1], width):
        part = v[:, at:at + width]
        amax = part.abs().max(1).values
        step = amax / 127.0
        safe = torch.where(amax > 0, amax, torch.ones_like(amax))[:, None]
        q[:, at:at + width] = torch.round(127.0 * part / safe)  # torch rounds halves to even
        scales.append(step)
    return q, torch.stack(scales, 1)


def _values_64(q, s, width):
    out = q.double().clone()
    for b in range(s.shape[1]):
        out[:, b * width:(b + 1) * width] *= s[:, b:b + 1].double()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize_rows":
        q, s = _codes_64(st["x"].double(), case["K"])
        return {"q": q.to(torch.int8), "scale": s[:, 0]}
    if op == "save_rows":
        q, s = _codes_64(st["x"].double(), SAVED)
        return {"q": q.to(torch.int8), "scale": s, "back": _values_64(q, s, SAVED)}
    if op == "gemm":
        out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        a = st["aq"].double() * st["a_scale"].double()[:, None]
        ends = st["offsets"].tolist()
        for e in range(case["E"]):
            if ends[e + 1] > ends[e]:
                w = st["wq"][e].double() * st["w_scale"][e].double()[:, None]
                out[ends[e]:ends[e + 1]] = a[ends[e]:ends[e + 1]] @ w.T
        return out if st["row_weight"] is None else out * st["row_weight"].double()[:, None]
    T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))

    def matrix(m, e):
        return m[0][e].double() * m[1][e].double()[:, None]

    if op in ("experts", "few"):
        x, logits = st["x"].double(), None
        if op == "few":
            logits = x @ st["w_router"].double().T + st["bias"].double()
            idx = torch.argsort(logits.float(), dim=1, descending=True, stable=True)[:, :k]
            p = torch.softmax(logits, 1).gather(1, idx)
            w = p / (p.sum(1, keepdim=True) + 1e-20)
        else:
            x = _values_64(*_codes_64(x, H), H)
            idx, w = st["topk_idx"].long(), st["topk_w"].double()
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for e in range(E):
            tok, slot = torch.nonzero(idx == e, as_tuple=True)
            if tok.numel() == 0:
                continue
            g, u = x[tok] @ matrix(st["gate"], e).T, x[tok] @ matrix(st["up"], e).T
            a = g * torch.sigmoid(g) * u
            if op == "experts":
                a = _values_64(*_codes_64(a, I), I)
            y.index_add_(0, tok, (a @ matrix(st["down"], e).T) * w[tok, slot][:, None])
        return y if op == "experts" else {"logits": logits, "idx": idx.to(torch.int32), "w": w, "y": y}
    ends = st["offsets"].tolist()
    tokens = st["row_token"].long()
    if op == "saved_forward":
        g = torch.zeros(T * k, I, dtype=torch.float64, device="cuda")
        u = torch.zeros_like(g)
        for e in range(E):
            rows = slice(ends[e], ends[e + 1])
            x = st["x"][tokens[rows]].double()
            g[rows], u[rows] = x @ st["w_gate"][e].double().T, x @ st["w_up"][e].double().T
        return {"a": g * torch.sigmoid(g) * u, "g": _values_64(*_codes_64(g, SAVED), SAVED),
                "u": _values_64(*_codes_64(u, SAVED), SAVED)}
    dA = torch.zeros(T * k, I, dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = slice(ends[e], ends[e + 1])
        dA[rows] = st["dy"][tokens[rows]].double() @ st["w_down"][e].double()
    g, u = _values_64(st["gq"], st["g_scale"], SAVED), _values_64(st["uq"], st["u_scale"], SAVED)
    w, sig = st["row_weight"].double()[:, None], torch.sigmoid(g)
    slope = sig + g * sig * (1.0 - sig)
    by_slot = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    by_slot[st["sorted_to_flat"].long()] = (dA * g * sig * u).sum(1)
    return {"dgu": torch.cat([w * dA * u * slope, w * dA * (g * sig)], 1), "a_w": w * g * sig * u,
            "d_topk_w": by_slot.view(T, k)}
