"""Cases for timing the operators around and inside the local experts in bf16
and in 8 bits: the root-mean-square norm that makes the rows a layer
dispatches (with its gradient), and the products grouped by expert, with their
gradients.

Rows in 8 bits are OCP e4m3fn: groups of 128 consecutive elements of a row
share a scale, amax / 448 in 32 bits (format "fp32") or the smallest power of
two p >= 2^-127 with 448 p >= amax ("ue8m0", the exponent bytes packed four to
a word, column-major).  Weights in 8 bits have one 32-bit scale for every block
of 128 x 128.

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the framework's calls.  The kinds of a case:

  norm    T rows of H elements: h = x + residual in bf16, y = h / sqrt(mean(h^2)
          + eps) * weight, as bf16 rows or as 8-bit rows (read back)
  normgrad  that norm and its gradient: dx (with the residual path's) and dweight
  fp8     rows of K elements against each expert's [N, K] weights, both 8 bits;
          rows in segments, or padded per expert (masked)
  experts8  dispatch in 8 bits, gate/up product with SwiGLU, down product, combine
  bf16    the product in bf16, or (swiglu) the gate/up product with SwiGLU
  train   one product's training pass: the product, or its SwiGLU form, and the
          gradients of the rows and of the weights
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
PACKED = 7                     # UE8M0 | COLMAJOR | PACKED of the framework's scale flags


def listed():
    return [
        # a decode batch before its expert layer: launch latency counts
        _norm("norm decode", T=128, H=7168, out="fp8", residual=True, fmt="ue8m0"),
        # a prefill step: 8-bit rows for the shared expert
        _norm("norm prefill", T=4096, H=7168, out="fp8", residual=True, fmt="fp32"),
        # training: ragged token count, a row width that is no power of two
        _normgrad("norm gradient ragged", T=4999, H=2592, residual=True),
        # training, a long batch
        _normgrad("norm gradient long", T=16384, H=4096, residual=True),
        # decode: a few rows an expert in the padded low-latency buffer, so the weights' bytes count
        _fp8("fp8 product decode", T=128, K=7168, N=4096, E=256, L=32, k=8, masked=True, fmt="ue8m0"),
        # the expert half of a prefill step in 8 bits, from token rows to token rows
        _experts8("fp8 experts prefill", T=4096, H=7168, I=2048, E=256, L=32, k=8, fmt="fp32"),
        # a long prefill with every expert local: the matrix rate counts
        _fp8("fp8 product long", T=16384, K=4096, N=4096, E=128, L=128, k=8, skew=0.3),
        # odd sizes, experts of unequal load
        _bf16("bf16 product ragged", T=1500, K=1440, N=5000, E=64, L=64, k=6, skew=0.5),
        # prefill, gate and up weights on one rank of eight
        _bf16("bf16 swiglu prefill", T=4096, K=7168, N=4096, E=256, L=32, k=8, swiglu=True),
        # a long prefill with every expert local
        _bf16("bf16 product long", T=16384, K=4096, N=4096, E=128, L=128, k=8, skew=0.3),
        # training on one rank of eight: the down product and its gradients
        _train("bf16 training", T=4096, K=2048, N=7168, E=256, L=32, k=8),
        # training, the gate/up product, odd sizes, experts of unequal load
        _train("bf16 swiglu training ragged", T=5000, K=2592, N=2112, E=40, L=40, k=6, skew=0.3, swiglu=True),
    ]


def _norm(name, T, H, out, residual, fmt="fp32"):
    return {"name": name, "kind": "norm", "T": T, "H": H, "out": out, "residual": residual, "fmt": fmt}


def _normgrad(name, T, H, residual):
    return {"name": name, "kind": "normgrad", "T": T, "H": H, "residual": residual}


def _fp8(name, T, K, N, E, L, k, skew=0.0, masked=False, fmt="fp32"):
    return {"name": name, "kind": "fp8", "T": T, "K": K, "N": N, "E": E, "L": L, "k": k, "skew": skew,
            "masked": masked, "fmt": fmt}


def _experts8(name, T, H, I, E, L, k, skew=0.0, align=1, fmt="fp32"):
    return {"name": name, "kind": "experts8", "T": T, "H": H, "I": I, "E": E, "L": L, "k": k, "skew": skew,
            "align": align, "fmt": fmt}


def _bf16(name, T, K, N, E, L, k, skew=0.0, masked=False, swiglu=False):
    return {"name": name, "kind": "bf16", "T": T, "K": K, "N": N, "E": E, "L": L, "k": k, "skew": skew,
            "masked": masked, "swiglu": swiglu}


def _train(name, T, K, N, E, L, k, skew=0.0, swiglu=False):
    return {"name": name, "kind": "train", "T": T, "K": K, "N": N, "E": E, "L": L, "k": k, "skew": skew,
            "swiglu": swiglu}


def draw(rng):
    """One more case: sizes spread over the logarithm of their ranges."""
    def size(lo, hi, step):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
        return min(hi, max(lo, int(v) // step * step))

    kind = rng.choice(["norm", "norm", "normgrad", "fp8", "fp8", "experts8", "bf16", "bf16", "train", "train"])
    fmt = rng.choice(["fp32", "ue8m0"])
    if kind == "norm":
        out = rng.choice(["fp8", "fp8", "bf16"])
        c = _norm("", size(1, 16384, 1), size(128, 7168, 128 if out == "fp8" else 1), out, rng.random() < 0.7, fmt)
    elif kind == "normgrad":
        c = _normgrad("", size(1, 16384, 1), size(64, 7168, rng.choice([1, 8])), rng.random() < 0.7)
    else:
        L = rng.choice([4, 8, 17, 32, 40, 64, 128 if kind in ("fp8", "bf16") else 24])
        E = L * rng.choice([1, 1, 2, 8])
        k = rng.randint(1, min(8, E))
        skew = rng.choice([0.0, 0.0, 0.3, 0.5]) if E == L else 0.0
        masked = kind in ("fp8", "bf16") and rng.random() < 0.35
        T = size(1, 512, 1) if masked else size(16, 16384 if kind in ("fp8", "bf16") else 4096, 1)
        if kind == "fp8":
            c = _fp8("", T, size(128, 7168, 128), size(128, 7168, 8), E, L, k, skew, masked, fmt)
        elif kind == "experts8":
            c = _experts8("", T, size(128, 7168, 128), size(128, 2048, 128), E, L, k, skew, rng.choice([1, 16, 128]), fmt)
        elif kind == "bf16":
            swiglu = rng.random() < 0.4
            c = _bf16("", T, size(64, 7168, 8), size(64, 7168, 16), E, L, k, skew, masked, swiglu)
        else:
            c = _train("", T, size(64, 4096, 8), size(64, 4096, 16), E, L, k, skew, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)


def _bf16_weights(g, L, n, m):
    w = torch.empty(L, n, m, device=DEV, dtype=torch.bfloat16)
    for e in range(L):
        w[e] = _normal(g, n, m, scale=m ** -0.5)
    return w


def _fp8_weights(g, L, n, m):
    """e4m3fn bytes [L, n, m] and the scales [L, ceil(n / 128), m / 128] of their blocks."""
    q = torch.empty(L, n, m, device=DEV, dtype=torch.uint8)
    s = torch.empty(L, (n + 127) // 128, m // 128, device=DEV)
    for e in range(L):
        w = torch.nn.functional.pad(_normal(g, n, m, scale=m ** -0.5), (0, 0, 0, -n % 128))
        b = w.view(-1, 128, m // 128, 128)
        s[e] = b.abs().amax((1, 3)) / 448
        q[e] = (b / s[e][:, None, :, None]).reshape(w.shape)[:n].to(torch.float8_e4m3fn).view(torch.uint8)
    return q, s


def _routing(case, g):
    """Distinct expert ids of every token and softmax weights."""
    T, E, k = case["T"], case["E"], case["k"]
    p = torch.arange(1, E + 1, device=DEV, dtype=torch.float32).pow(-case["skew"])
    p = p[torch.randperm(E, generator=g, device=DEV)] if case["skew"] else p
    ids = torch.multinomial(p.expand(T, E), k, replacement=False, generator=g).to(torch.int32)
    return ids, torch.softmax(_normal(g, T, k), -1)


def _rows(case):
    """Rows of a program's fixed buffers: every slot where all experts are local (with the segments' padding),
    otherwise the expected number and six standard deviations."""
    n, pad = case["T"] * min(case["k"], case["L"]), case["L"] * (case.get("align", 1) - 1)
    if case["E"] > case["L"]:
        mean = case["T"] * case["k"] * case["L"] / case["E"]
        n = min(n, int(mean + 6 * math.sqrt(mean)) + 8)
    return n + pad


def _flags(case):
    return PACKED if case["fmt"] == "ue8m0" else 0


def _in_format(s, fmt):
    """Scales s [mats, rows, G] as the framework's buffers hold them."""
    if fmt == "fp32":
        return s
    mats, rows, G = s.shape
    ld = (rows + 3) // 4 * 4
    code = torch.zeros(mats, (G + 3) // 4 * 4, ld, device=s.device, dtype=torch.int64)
    code[:, :G, :rows] = (torch.frexp(s)[1] + 126).transpose(1, 2)      # s = 0.5 * 2^exponent
    b = code.view(mats, -1, 4, ld)
    word = b[:, :, 0] | b[:, :, 1] << 8 | b[:, :, 2] << 16 | b[:, :, 3] << 24
    return torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)


def _scale_values(t, fmt, rows, G):
    """fp32 scales [mats, rows, G] of a buffer of _in_format."""
    if fmt == "fp32":
        return t
    b = torch.stack([t >> (8 * i) & 255 for i in range(4)], 2).flatten(1, 2)[:, :G, :rows]
    return torch.ldexp(torch.ones_like(b, dtype=torch.float32), b - 127).transpose(1, 2)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    T, kind = case["T"], case["kind"]
    if kind in ("norm", "normgrad"):
        H = case["H"]
        s = {"case": case, "x": _normal(g, T, H, dtype=torch.bfloat16),
             "weight": (1 + _normal(g, H, scale=0.1)).to(torch.bfloat16),
             "residual": _normal(g, T, H, scale=4.0, dtype=torch.bfloat16) if case["residual"] else None}
        if kind == "normgrad":
            s["dy"] = _normal(g, T, H, scale=0.01, dtype=torch.bfloat16)
            s["dh"] = _normal(g, T, H, scale=0.01, dtype=torch.bfloat16) if case["residual"] else None
        return s
    ids, weights = _routing(case, g)
    L = case["L"]
    counts, seg, dst = _layout(ids, L, case.get("align", 1))
    rows = _rows(case)
    s = {"case": case, "ids": ids, "weights": weights, "rows": rows, "counts": counts, "seg": seg,
         "most": max(1, int(counts.max()))}
    if kind == "experts8":
        s["x"] = _normal(g, T, case["H"], dtype=torch.bfloat16)
        s["w13"] = _fp8_weights(g, L, 2 * case["I"], case["H"])
        s["w2"] = _fp8_weights(g, L, case["H"], case["I"])
        return s
    K, N = case["K"], case["N"]
    masked = case.get("masked", False)
    lead = (L, T) if masked else (1, rows)                  # a token goes to an expert at most once
    a = _normal(g, *lead, K, dtype=torch.bfloat16)
    if kind == "fp8":
        s["w"] = _fp8_weights(g, L, N, K)
        r, p = _rounded(a.float(), case["fmt"])
        q = r.to(torch.float8_e4m3fn).view(torch.uint8)
        s["a"] = (q if masked else q[0], _in_format(p, case["fmt"]))
        if not masked and case["fmt"] == "fp32":
            s["a"] = (s["a"][0], s["a"][1][0])
    else:
        s["w"] = _bf16_weights(g, L, N, K)
        s["a"] = a if masked else a[0]
    wide = N // 2 if case.get("swiglu") else N
    # rows of no expert are never written: the buffers a program keeps start as zeros
    s["out"] = torch.zeros(*(lead if masked else lead[1:]), wide, device=DEV, dtype=torch.bfloat16)
    if kind == "train":
        s["dy"] = _normal(g, rows, wide, scale=0.01, dtype=torch.bfloat16)
        s["dgu"] = torch.zeros(rows, N, device=DEV, dtype=torch.bfloat16) if case["swiglu"] else None
        s["dx"] = torch.zeros(rows, K, device=DEV, dtype=torch.bfloat16)
        s["dw"] = torch.zeros(L, N, K, device=DEV, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _own(case["kind"], case, s)
    return {"norm": _plain_norm, "normgrad": _plain_normgrad, "fp8": _plain_fp8, "experts8": _plain_experts8,
            "bf16": _plain_bf16, "train": _plain_train}[case["kind"]](case, s)


def _own(kind, case, s):
    import combine_dispatch_layout_amd as cdl

    if kind == "norm":
        if case["out"] == "bf16":
            got = cdl.rms_norm(s["x"], s["weight"], s["residual"], EPS)
            return {"y": got[0], "h": got[1]} if case["residual"] else {"y": got}
        got = cdl.rms_norm_fp8(s["x"], s["weight"], s["residual"], EPS, scale_flags=_flags(case))
        y = cdl.dequant_fp8(got[0], got[1], scale_flags=_flags(case))
        return {"y": y, "h": got[2]} if case["residual"] else {"y": y}
    if kind == "normgrad":
        if case["residual"]:
            y, h = cdl.rms_norm(s["x"], s["weight"], s["residual"], EPS)
        else:
            y, h = cdl.rms_norm(s["x"], s["weight"], None, EPS), s["x"]
        dx, dweight = cdl.rms_norm_grad(s["dy"], h, s["weight"], EPS, s["dh"])
        return {"y": y, "dx": dx, "dweight": dweight}
    if kind == "fp8":
        seg = None if case["masked"] else s["seg"]
        return cdl.grouped_fp8(*s["a"], *s["w"], s["counts"], seg, scale_flags=_flags(case), out=s["out"])
    if kind == "experts8":
        f = _flags(case)
        lay, q, sc = cdl.permute_fp8(s["x"], s["ids"], 0, case["L"], rows=s["rows"], alignment=case["align"],
                                     scale_flags=f)
        h, hs = cdl.grouped_swiglu_fp8(q, sc, *s["w13"], lay.counts, lay.seg_indptr, scale_flags=f)
        y = cdl.grouped_fp8(h, hs, *s["w2"], lay.counts, lay.seg_indptr, scale_flags=f)
        return cdl.combine(y, lay.src2dst, s["weights"])
    if kind == "bf16":
        seg = None if case["masked"] else s["seg"]
        product = cdl.grouped_swiglu_bf16 if case["swiglu"] else cdl.grouped_bf16
        return product(s["a"], s["w"], s["counts"], seg, out=s["out"])
    at = (s["counts"], s["seg"])
    if case["swiglu"]:
        y = cdl.grouped_swiglu_bf16(s["a"], s["w"], *at, out=s["out"])
        dy = cdl.grouped_swiglu_bf16_grad(s["a"], s["w"], s["dy"], *at, out=s["dgu"])
    else:
        y = cdl.grouped_bf16(s["a"], s["w"], *at, out=s["out"])
        dy = s["dy"]
    dx = cdl.grouped_bf16_dx(dy, s["w"], *at, out=s["dx"])
    dw = cdl.grouped_bf16_dw(dy, s["a"], *at, out=s["dw"])
    return {"y": y, "dx": dx, "dw": dw, **({"dgu": dy} if case["swiglu"] else {})}


def _layout(ids, L, align):
    """counts [L], seg_indptr [L + 1] and the destination row of every slot (-1: not local)."""
    n = ids.numel()
    e = ids.reshape(-1).long()
    key = torch.where((e >= 0) & (e < L), e, L)
    counts = torch.zeros(L + 1, device=ids.device, dtype=torch.int64).scatter_add_(0, key, torch.ones_like(key))
    padded = (counts[:L] + align - 1) // align * align
    seg = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    order = torch.argsort(key, stable=True)
    first = counts.cumsum(0) - counts                        # of each expert in the sorted order
    at = torch.arange(n, device=ids.device)
    sorted_key = key[order]
    dst = torch.cat([seg[:L], seg.new_zeros(1)])[sorted_key] + at - first[sorted_key]
    src2dst = torch.empty_like(key)
    src2dst[order] = torch.where(sorted_key < L, dst, -1)
    return counts[:L].to(torch.int32), seg, src2dst.to(torch.int32)


def _group_scale(v, fmt):
    """The scale of every group of 128 of v [..., m]."""
    top = v.unflatten(-1, (-1, 128)).abs().amax(-1)
    if fmt == "fp32":
        return (top.double() / 448).float()
    m, e = torch.frexp(top)                                  # 448 = 0.875 * 2^9
    e = torch.where(top == 0, -127, torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-127))
    return torch.ldexp(torch.ones_like(top), e)


def _rounded(v, fmt):
    """(e4m3fn values [..., m] in 32 bits, scales [..., m / 128]) of v [..., m]."""
    p = _group_scale(v, fmt)
    # divided in 64 bits, then rounded to 32: bf16 values often fall halfway between two codes
    t = (v.unflatten(-1, (-1, 128)).double() / torch.where(p == 0, 1, p).double().unsqueeze(-1)).float()
    return t.clamp(-448, 448).flatten(-2).to(torch.float8_e4m3fn).float(), p


def _quantised(v, fmt):
    """The values that v [..., m] stands for in 8 bits."""
    r, p = _rounded(v, fmt)
    return (r.unflatten(-1, (-1, 128)) * p.unsqueeze(-1)).flatten(-2)


def _plain_sum(s):
    h = s["x"].float()
    return h if s["residual"] is None else (h + s["residual"].float()).to(torch.bfloat16).float()


def _plain_norm(case, s):
    h = _plain_sum(s)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if case["out"] == "fp8":
        y = _quantised(y, case["fmt"])
    y = y.to(torch.bfloat16)
    return {"y": y, "h": h.to(torch.bfloat16)} if case["residual"] else {"y": y}


def _plain_normgrad(case, s):
    h, dy, w = _plain_sum(s), s["dy"].float(), s["weight"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n = h * r
    d = dy * w
    dx = r * (d - n * (d * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"y": (n * w).to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dweight": (dy * n).sum(0)}


def _fp8_values(q):
    return q.view(torch.float8_e4m3fn).float()


def _weight_values(q, s):
    """fp32 values [L, n, m] of weights in blocks of 128 x 128."""
    w = _fp8_values(q).unflatten(-1, (-1, 128))
    return w.mul_(s.repeat_interleave(128, 1)[:, :q.shape[1]].unsqueeze(-1)).flatten(-2)


def _row_values(q, s, fmt):
    """fp32 values of 8-bit rows q [..., m]."""
    v = _fp8_values(q).unflatten(-1, (-1, 128))
    p = _scale_values(s, fmt, q.shape[-2], q.shape[-1] // 128).view(v.shape[:-1])
    return v.mul_(p.unsqueeze(-1)).flatten(-2)


def _padded(a, seg, most):
    """Rows a [R, K] in segments as [L, most, K]."""
    at = (seg[:-1, None] + torch.arange(most, device=a.device)).clamp(max=a.shape[0] - 1)
    return a[at]


def _live(counts, most):
    return (torch.arange(most, device=counts.device) < counts[:, None]).unsqueeze(-1)


def _in_rows(y, counts, seg, R):
    """y [L, most, N] as rows [R, N] in segments; rows behind an expert's count are 0."""
    r = torch.arange(R, device=y.device)
    e = torch.searchsorted(seg[1:], r, right=True).clamp(max=y.shape[0] - 1)
    m = r - seg[e]
    return torch.where((m < counts[e]).unsqueeze(1), y[e, m.clamp(min=0, max=y.shape[1] - 1)], 0.0)


def _grouped(a, w, counts, seg, most):
    """fp32 products of the rows a [R, K] in segments with w [L, N, K]."""
    y = torch.bmm(_padded(a, seg, most), w.transpose(1, 2).contiguous())
    return _in_rows(y, counts, seg, a.shape[0])


def _swiglu(gu):
    g, u = gu.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def _product(case, s, a, w):
    """The product's bf16 rows in the state's buffer."""
    counts = s["counts"].long()
    if not case.get("masked"):
        y = _grouped(a, w, counts, s["seg"], s["most"])
        s["out"].copy_(_swiglu(y) if case.get("swiglu") else y)
        return s["out"]
    y = torch.bmm(a[:, :s["most"]], w.transpose(1, 2).contiguous())
    y = _swiglu(y) if case.get("swiglu") else y
    s["out"][:, :s["most"]] = torch.where(_live(counts, s["most"]), y, 0.0).to(torch.bfloat16)
    return s["out"]


def _plain_fp8(case, s):
    return _product(case, s, _row_values(*s["a"], case["fmt"]), _weight_values(*s["w"]))


def _plain_bf16(case, s):
    return _product(case, s, s["a"].float(), s["w"].float())


def _plain_experts8(case, s):
    T, k, fmt = case["T"], case["k"], case["fmt"]
    counts, seg, dst = _layout(s["ids"], case["L"], case["align"])
    counts, valid = counts.long(), dst >= 0
    rows = s["rows"]
    a = s["x"].new_zeros(rows + 1, case["H"], dtype=torch.float32)
    a.index_copy_(0, torch.where(valid, dst, rows).long(), _quantised(s["x"].float(), fmt).repeat_interleave(k, 0))
    h = _swiglu(_grouped(a[:rows], _weight_values(*s["w13"]), counts, seg, s["most"]))
    y = _grouped(_quantised(h, fmt), _weight_values(*s["w2"]), counts, seg, s["most"])
    wt = torch.where(valid, s["weights"].reshape(-1), 0.0).unsqueeze(1)
    return (y[dst.clamp(min=0).long()] * wt).view(T, k, -1).sum(1).to(torch.bfloat16)


def _plain_train(case, s):
    counts, seg, most = s["counts"].long(), s["seg"], s["most"]
    R = s["rows"]
    live = _live(counts, most)
    w = s["w"].float()
    a = torch.where(live, _padded(s["a"].float(), seg, most), 0.0)
    dy = torch.where(live, _padded(s["dy"].float(), seg, most), 0.0)
    y = torch.bmm(a, w.transpose(1, 2).contiguous())
    if case["swiglu"]:
        g, u = y.chunk(2, -1)
        sg = 1 / (1 + torch.exp(-g))
        y = g * sg * u
        # the gradient of the gate and up values, in the type of the products that take it
        dy = torch.cat([dy * u * sg * (1 + g * (1 - sg)), dy * g * sg], -1).to(torch.bfloat16).float()
        s["dgu"].copy_(_in_rows(dy, counts, seg, R))
    s["out"].copy_(_in_rows(y, counts, seg, R))
    s["dx"].copy_(_in_rows(torch.bmm(dy, w), counts, seg, R))
    s["dw"].copy_(torch.bmm(dy.transpose(1, 2).contiguous(), a))
    return {"y": s["out"], "dx": s["dx"], "dw": s["dw"], **({"dgu": s["dgu"]} if case["swiglu"] else {})}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    T, kind = case["T"], case["kind"]
    if kind in ("norm", "normgrad"):
        n, res = T * case["H"], 1 if case["residual"] else 0
        if kind == "normgrad":
            return {"bytes": n * (2 + 2 + 2 * res) + n * (2 + 2 + 2 * res) + 6 * case["H"], "flops": 0}
        q = 1 + 4 / 128 if case["fmt"] == "fp32" else 1 + 1 / 128
        return {"bytes": n * (2 + 4 * res) + (n * (2 * q + 2) if case["out"] == "fp8" else n * 2) + 2 * case["H"],
                "flops": 0}
    E, L, k = case["E"], case["L"], case["k"]
    R = T * k * L / E                                            # expected local slots
    active = L * (1 - (1 - k / E) ** T)                          # experts with one
    if kind == "experts8":
        H, I = case["H"], case["I"]
        U = T * (1 - math.prod((E - L - j) / (E - j) for j in range(k)))  # tokens with a local slot
        return {"bytes": T * k * 8 + U * H * 2 + active * 3 * I * H + T * H * 2, "flops": 6 * R * H * I}
    K, N = case["K"], case["N"]
    wide = N // 2 if case.get("swiglu") else N
    if kind == "train":
        extra = 2 * R * N if case["swiglu"] else 0               # the gate and up gradients
        return {"bytes": 2 * (2 * R * K + 2 * R * wide + active * N * K + L * N * K) + extra,
                "flops": (4 if case["swiglu"] else 3) * 2 * R * K * N}
    each = 2 if kind == "bf16" else 1
    return {"bytes": R * K * each + active * N * K * each + R * wide * 2, "flops": 2 * R * K * N}


def _exact_bytes(q):
    """Values of e4m3fn bytes in 64 bits."""
    c = q.long()
    ex, man = c >> 3 & 15, (c & 7).double()
    mag = torch.where(ex == 0, man * 2.0 ** -9, (8 + man) * torch.pow(2.0, (ex - 10).double()))
    return torch.where(c >= 128, -mag, mag)


def _exact_quantised(v, fmt):
    """8-bit values of v [rows, m] in 64 bits: the nearest e4m3fn value, halfway to the even code.  The format's
    scale and the quotient by it are 32-bit numbers by definition."""
    b = v.double().reshape(v.shape[0], -1, 128)
    top = b.abs().amax(-1, keepdim=True)
    if fmt == "fp32":
        p = (top / 448).float().double()
    else:
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448))
        e = torch.where(448 * torch.pow(2.0, e - 1) >= top, e - 1, e)
        e = torch.where(448 * torch.pow(2.0, e) < top, e + 1, e).clamp(min=-127)
        p = torch.where(top > 0, torch.pow(2.0, e), 2.0 ** -127)
    t = (b / torch.where(p > 0, p, 1.0)).float().double()
    # the spacing of e4m3fn at t: 2^(exponent - 3), 2^-9 below 2^-6; torch.round takes halves to the even multiple
    step = torch.pow(2.0, torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return ((torch.round(t / step) * step).clamp(-448, 448) * p).reshape(v.shape)


def _exact_scales(t, fmt, m, rows, G):
    """Scales [rows, G] of matrix m of a buffer."""
    if fmt == "fp32":
        return t.reshape(-1, G)[m * rows:(m + 1) * rows].double()
    b = t[m].contiguous().view(torch.uint8).view(t.shape[1], t.shape[2], 4).permute(0, 2, 1).reshape(-1, t.shape[2])
    return torch.pow(2.0, b[:G, :rows].t().double() - 127)


def _exact_weights(q, s, e):
    n, m = q.shape[1:]
    block = torch.arange(n, device=q.device) // 128
    return (_exact_bytes(q[e]).reshape(n, -1, 128) * s[e].double()[block].unsqueeze(-1)).reshape(n, m)


def _exact_swiglu(gu):
    gate, up = gu.split(gu.shape[-1] // 2, -1)
    return gate * torch.sigmoid(gate) * up


def _exact_norm(case, s):
    h = s["x"].double()
    if case["residual"]:
        h = (h + s["residual"].double()).to(torch.bfloat16).double()
    w = s["weight"].double()
    size = torch.sqrt(h.pow(2).sum(-1, keepdim=True) / case["H"] + EPS)
    y = h / size * w
    if case["kind"] == "norm":
        y = _exact_quantised(y, case["fmt"]) if case["out"] == "fp8" else y
        return {"y": y, "h": h} if case["residual"] else {"y": y}
    dy = s["dy"].double()
    inner = (dy * w * h).sum(-1, keepdim=True)
    dx = dy * w / size - h * inner / (case["H"] * size.pow(3))
    if case["residual"]:
        dx = dx + s["dh"].double()
    return {"y": y, "dx": dx, "dweight": (dy * h / size).sum(0)}


def exact(case, seed):
    s = prepare(case, seed)
    kind, T, L = case["kind"], case["T"], case["L"] if "L" in case else 0
    if kind in ("norm", "normgrad"):
        return _exact_norm(case, s)
    counts = s["counts"].tolist()
    if kind == "experts8":
        k, fmt = case["k"], case["fmt"]
        ids, w = s["ids"].reshape(-1), s["weights"].reshape(-1).double()
        token = torch.arange(T, device=DEV).repeat_interleave(k)
        a = _exact_quantised(s["x"], fmt)
        out = torch.zeros(T, case["H"], device=DEV, dtype=torch.float64)
        for e in range(L):
            at = (ids == e).nonzero().reshape(-1)
            if len(at):
                h = _exact_quantised(_exact_swiglu(a[token[at]] @ _exact_weights(*s["w13"], e).t()), fmt)
                out.index_add_(0, token[at], (h @ _exact_weights(*s["w2"], e).t()) * w[at].unsqueeze(1))
        return out
    K, masked = case["K"], case.get("masked", False)
    first = [e * T for e in range(L)] if masked else s["seg"].tolist()
    out = torch.zeros(s["out"].numel() // s["out"].shape[-1], s["out"].shape[-1], device=DEV, dtype=torch.float64)
    grads = None
    if kind == "train":
        grads = {"dx": torch.zeros(s["rows"], K, device=DEV, dtype=torch.float64),
                 "dw": torch.zeros(L, case["N"], K, device=DEV, dtype=torch.float64)}
        if case["swiglu"]:
            grads["dgu"] = torch.zeros(s["rows"], case["N"], device=DEV, dtype=torch.float64)
    for e in range(L):
        n = counts[e]
        if not n:
            continue
        at = slice(first[e], first[e] + n)
        if kind == "fp8":
            q, sc = s["a"]
            q = q.reshape(-1, K)
            p = (_exact_scales(sc, case["fmt"], e, T, K // 128)[:n] if masked
                 else _exact_scales(sc, case["fmt"], 0, q.shape[0], K // 128)[at])
            a = (_exact_bytes(q[at]).reshape(n, -1, 128) * p.unsqueeze(-1)).reshape(n, K)
            w = _exact_weights(*s["w"], e)
        else:
            a, w = s["a"].reshape(-1, K)[at].double(), s["w"][e].double()
        y = a @ w.t()
        out[at] = _exact_swiglu(y) if case.get("swiglu") else y
        if kind == "train":
            dy = s["dy"][at].double()
            if case["swiglu"]:
                gate, up = y.split(case["N"] // 2, -1)
                sg = torch.sigmoid(gate)
                dy = torch.cat([dy * up * (sg + gate * sg * (1 - sg)), dy * gate * sg], -1)
                grads["dgu"][at] = dy
                dy = dy.to(torch.bfloat16).double()          # the type of the products that take it
            grads["dx"][at] = dy @ w
            grads["dw"][e] = dy.t() @ a
    if kind == "train":
        return {"y": out, **grads}
    return out.view(s["out"].shape)
