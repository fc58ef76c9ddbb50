"""The 8-bit integer operators (include/moe_i8.h, include/moe_ckpt8.h) in 64 bits, on
the CPU: codes with one scale per row or per 64 columns, the grouped product, the
expert stage, and the backward of the down projection from kept activations."""
import torch

BLOCK = 64


def codes(v, width=None):
    """v [R,K] -> (codes [R,K] int8, scales [R,ceil(K/width)] float64); one scale per row without width.
    A block with a NaN or an infinity: codes 0, scale NaN."""
    v = v.double()
    R, K = v.shape
    width = K if width is None else width
    n = -(-K // width)
    p = torch.cat([v, v.new_zeros(R, n * width - K)], 1).view(R, n, width)
    amax = p.abs().amax(2)
    fine = p.isfinite().all(2)
    safe = torch.where(fine & (amax > 0), amax, torch.ones_like(amax))
    q = torch.where(fine[:, :, None] & (amax > 0)[:, :, None], torch.round(127.0 * p / safe[:, :, None]), torch.zeros_like(p))
    scale = torch.where(fine, amax / 127.0, torch.full_like(amax, float("nan")))
    return q.to(torch.int8).view(R, -1)[:, :K].contiguous(), scale


def values(q, scale):
    K = q.shape[1]
    width = K if scale.shape[1] == 1 else BLOCK
    return q.double() * scale.double().repeat_interleave(width, 1)[:, :K]


def weights(w):
    """w [E,N,K] -> codes [E,N,K], scale [E,N]."""
    E, N, K = w.shape
    q, s = codes(w.reshape(E * N, K))
    return q.view(E, N, K), s.view(E, N)


def weight_values(q, scale):
    return q.double() * scale.double()[:, :, None]


def product(aq, sa, offsets, wq, sw, row_weight=None):
    out = torch.full((aq.shape[0], wq.shape[1]), float("nan"), dtype=torch.float64)
    for e in range(wq.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        sums = aq[r].double() @ wq[e].double().T
        out[r] = sums * sa[r].double()[:, None] * sw[e].double()[None]
    return out if row_weight is None else out * row_weight.double()[:, None]


def experts(x, idx, w, gate, up, down, near=0.0):
    """y [T,H] of the expert stage on (codes, scales) weights, and how far each output may be off
    where codes of a that lie within `near` steps of a border fall on its other side."""
    T, k = idx.shape
    E = gate[0].shape[0]
    xv = values(*codes(x))
    y = torch.zeros(T, down[0].shape[1], dtype=torch.float64)
    slack, size = torch.zeros_like(y), torch.zeros_like(y)
    for e in range(E):
        tok, slot = torch.nonzero(idx == e, as_tuple=True)
        if tok.numel() == 0:
            continue
        g = xv[tok] @ weight_values(*gate)[e].T
        u = xv[tok] @ weight_values(*up)[e].T
        a = g * torch.sigmoid(g) * u
        q, s = codes(a)
        wd = weight_values(*down)[e]
        pw = w[tok, slot].double()[:, None]
        y.index_add_(0, tok, pw * (values(q, s) @ wd.T))
        size.index_add_(0, tok, (pw * (values(q, s) @ wd.T)).abs())
        steps = a / torch.where(s > 0, s, torch.ones_like(s))
        edge = ((steps - torch.floor(steps)) - 0.5).abs() < near
        slack.index_add_(0, tok, pw.abs() * ((edge * s) @ wd.abs().T))
    return y, slack, size


def down_backward(dy, row_token, row_weight, offsets, w_down, gv, uv):
    """(dgu, a_w, d per sorted row) from the kept activations' values gv, uv [M,I]."""
    M, I = gv.shape
    dA = torch.zeros(M, I, dtype=torch.float64)
    for e in range(w_down.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        dA[r] = dy[row_token[r].long()].double() @ w_down[e].double()
    s = torch.sigmoid(gv)
    a = gv * s * uv
    w = row_weight.double()[:, None]
    dgu = torch.cat([w * dA * uv * s * (1.0 + gv * (1.0 - s)), w * dA * gv * s], 1)
    return dgu, w * a, (dA * a).sum(1)
