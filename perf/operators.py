"""Cases for timing the expert operators: MXFP4 rows on the scatter, the
grouped MXFP4 product of the local experts, the whole expert step in MXFP4,
and the MoE layer of a few tokens.

MXFP4 (OCP microscaling, e2m1 elements): groups of 32 consecutive elements
share one scale 2^e, stored as the byte e + 127; an element is 4 bits (sign,
two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a
byte, the even element in the low half.  e is the smallest integer >= -127
with 6 * 2^e >= the group's largest magnitude; elements round to nearest, ties
to the even code.

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the framework's calls.  The kinds of a case:

  dispatch  T tokens of H elements: routing layout, the rows of the L local of
            E experts quantised on the scatter, and read back
  product   rows of K elements against each expert's [N, K] weights, both
            MXFP4; rows in segments, or padded per expert (masked)
  experts   dispatch, gate/up product with SwiGLU, down product, combine
  layer     the experts of a few tokens from bf16 rows, in bf16 or MXFP4 weights
"""
import math

import torch

own = False

DEV = "cuda"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the smallest batch of the parity configuration: launch latency counts
        _dispatch("dispatch tiny", T=64, H=256, E=8, L=8, k=2),
        # one rank of eight in a prefill step
        _dispatch("dispatch prefill", T=4096, H=7168, E=256, L=32, k=8),
        # skewed routing, a row width that is no power of two, padded segments
        _dispatch("dispatch skewed ragged", T=4999, H=2592, E=128, L=128, k=8, skew=1.2, align=16),
        # decode: a few rows an expert in the padded low-latency buffer, so the weights' bytes count
        _product("product decode", T=128, K=7168, N=4096, E=256, L=32, k=8, masked=True),
        # prefill, gate and up weights: about 128 rows an expert
        _product("product prefill", T=4096, K=7168, N=4096, E=256, L=32, k=8),
        # odd sizes in a down product, experts of unequal load
        _product("product ragged", T=1500, K=1440, N=5000, E=64, L=64, k=6, skew=0.5),
        # a long prefill with every expert local: the matrix rate counts
        _product("product long", T=16384, K=4096, N=4096, E=128, L=128, k=8, skew=0.3),
        # the expert half of a prefill step, from token rows to token rows
        _experts("experts prefill", T=4096, H=7168, I=2048, E=256, L=32, k=8),
        # one new token of a single sequence, every expert local
        _layer("layer one token", T=1, H=7168, I=2048, E=32, L=32, k=8, weights="bf16"),
        # a decode batch on one rank of eight
        _layer("layer decode batch", T=128, H=7168, I=2048, E=256, L=32, k=8, weights="bf16"),
        # the same single token with 4-bit weights
        _layer("layer one token mxfp4", T=1, H=7168, I=2048, E=32, L=32, k=8, weights="mxfp4"),
        # a ragged batch, odd sizes, 4-bit weights
        _layer("layer ragged mxfp4", T=37, H=2592, I=1056, E=40, L=40, k=6, weights="mxfp4"),
    ]


def _dispatch(name, T, H, E, L, k, skew=0.0, align=1):
    return {"name": name, "kind": "dispatch", "T": T, "H": H, "E": E, "L": L, "k": k, "skew": skew, "align": align}


def _product(name, T, K, N, E, L, k, skew=0.0, masked=False):
    return {"name": name, "kind": "product", "T": T, "K": K, "N": N, "E": E, "L": L, "k": k, "skew": skew,
            "masked": masked}


def _experts(name, T, H, I, E, L, k, skew=0.0, align=1):
    return {"name": name, "kind": "experts", "T": T, "H": H, "I": I, "E": E, "L": L, "k": k, "skew": skew,
            "align": align}


def _layer(name, T, H, I, E, L, k, weights, skew=0.0):
    return {"name": name, "kind": "layer", "T": T, "H": H, "I": I, "E": E, "L": L, "k": k, "skew": skew,
            "weights": weights}


def draw(rng):
    """One more case: sizes spread over the logarithm of their ranges."""
    def size(lo, hi, step):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
        return min(hi, max(lo, int(v) // step * step))

    kind = rng.choice(["dispatch", "product", "product", "experts", "layer", "layer"])
    L = rng.choice([4, 8, 17, 32, 40, 64, 128 if kind in ("dispatch", "product") else 24])
    E = L * rng.choice([1, 1, 2, 8])
    k = rng.randint(1, min(8, E))
    skew = rng.choice([0.0, 0.0, 0.3, 0.5]) if E == L else 0.0
    if kind == "dispatch":
        T, H = size(64, 16384, 1), size(256, 7168, 32)
        T = min(T, max(64, int(4096 * 7168 * 8 / (H * k))))
        c = _dispatch("", T, H, E, L, k, rng.choice([0.0, 0.3, 1.2]) if E == L else 0.0, rng.choice([1, 1, 16, 128]))
    elif kind == "product":
        K, N = size(256, 7168, 32), size(256, 7168, 8)
        masked = rng.random() < 0.4
        T = size(32, 512, 1) if masked else size(64, 16384, 1)
        c = _product("", T, K, N, E, L, k, skew, masked)
    elif kind == "experts":
        H, I = size(256, 7168, 32), size(128, 2048, 32)
        c = _experts("", size(64, 4096, 1), H, I, E, L, k, skew, rng.choice([1, 16]))
    else:
        H, I = size(256, 7168, 32), size(128, 2048, 32)
        c = _layer("", size(1, 128, 1), H, I, E, L, k, rng.choice(["bf16", "mxfp4"]), skew)
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


def _mxfp4_weights(g, L, n, m):
    q = torch.empty(L, n, m // 2, device=DEV, dtype=torch.uint8)
    s = torch.empty(L, n, m // 32, device=DEV, dtype=torch.uint8)
    for e in range(L):
        q[e], s[e] = _pack(_normal(g, n, m, scale=m ** -0.5))
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


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    ids, weights = _routing(case, g)
    T, L, k = case["T"], case["L"], case["k"]
    counts, seg, dst = _layout(ids, L, case.get("align", 1))
    rows = _rows(case)
    s = {"case": case, "ids": ids, "weights": weights, "rows": rows, "most": max(1, int(counts.max()))}
    if case["kind"] != "product":
        s["x"] = _normal(g, T, case["H"], dtype=torch.bfloat16)
    if case["kind"] == "dispatch":
        # padding rows are never written: the buffers a program keeps start as zeros
        s["q"] = torch.zeros(rows, case["H"] // 2, device=DEV, dtype=torch.uint8)
        s["scales"] = torch.zeros(rows, case["H"] // 32, device=DEV, dtype=torch.uint8)
    elif case["kind"] == "product":
        K, N = case["K"], case["N"]
        s["w"] = _mxfp4_weights(g, L, N, K)
        s["counts"] = counts
        if case["masked"]:
            s["a"] = _pack(_normal(g, L, T, K))             # a token goes to an expert at most once
            s["out"] = torch.zeros(L, T, N, device=DEV, dtype=torch.bfloat16)
        else:
            s["a"] = _pack(_normal(g, rows, K))
            s["out"] = torch.zeros(rows, N, device=DEV, dtype=torch.bfloat16)
            s["seg"] = seg
    elif case["kind"] == "experts" or case["weights"] == "mxfp4":
        s["w13"] = _mxfp4_weights(g, L, 2 * case["I"], case["H"])
        s["w2"] = _mxfp4_weights(g, L, case["H"], case["I"])
    else:
        s["w13"] = _bf16_weights(g, L, 2 * case["I"], case["H"])
        s["w2"] = _bf16_weights(g, L, case["H"], case["I"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _own(case["kind"], case, s)
    return {"dispatch": _plain_dispatch, "product": _plain_product, "experts": _plain_experts,
            "layer": _plain_layer}[case["kind"]](case, s)


def _own(kind, case, s):
    import combine_dispatch_layout_amd as cdl

    L = case["L"]
    if kind == "dispatch":
        lay, q, sc = cdl.permute_mxfp4(s["x"], s["ids"], 0, L, out_q=s["q"], out_scales=s["scales"],
                                       alignment=case["align"])
        return {"rows": cdl.dequant_mxfp4(q, sc), "src2dst": lay.src2dst, "counts": lay.counts}
    if kind == "product":
        if case["masked"]:
            return cdl.grouped_mxfp4(*s["a"], *s["w"], s["counts"], out=s["out"])
        return cdl.grouped_mxfp4(*s["a"], *s["w"], s["counts"], s["seg"], out=s["out"])
    if kind == "experts":
        lay, q, sc = cdl.permute_mxfp4(s["x"], s["ids"], 0, L, rows=s["rows"], alignment=case["align"])
        h, hs = cdl.grouped_swiglu_mxfp4(q, sc, *s["w13"], lay.counts, lay.seg_indptr)
        y = cdl.grouped_mxfp4(h, hs, *s["w2"], lay.counts, lay.seg_indptr)
        return cdl.combine(y, lay.src2dst, s["weights"])
    if case["weights"] == "mxfp4":
        return cdl.moe_layer_mxfp4(s["x"], s["ids"], s["weights"], *s["w13"], *s["w2"])
    return cdl.moe_layer(s["x"], s["ids"], s["weights"], s["w13"], s["w2"])


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


def _exponent(v):
    """e of every group of 32 of v [..., m]: the smallest >= -127 with 6 * 2^e >= the largest magnitude."""
    m, e = torch.frexp(v.unflatten(-1, (-1, 32)).abs().amax(-1))
    return torch.where(m == 0, -127, torch.clamp(e - 3 + (m > 0.75).to(e.dtype), min=-127))


def _rounded(v):
    """(magnitudes on the e2m1 grid [..., groups, 32], exponents) of v [..., m]."""
    e = _exponent(v)
    t = torch.ldexp(v.unflatten(-1, (-1, 32)).abs(), -e.unsqueeze(-1))
    r = torch.where(t < 2, torch.round(2 * t) * 0.5, torch.where(t < 4, torch.round(t), torch.round(t * 0.5) * 2))
    return r, e


def _quantised(v):
    """The values that v [..., m] stands for in MXFP4."""
    r, e = _rounded(v)
    return torch.copysign(torch.ldexp(r, e.unsqueeze(-1)), v.unflatten(-1, (-1, 32))).flatten(-2)


def _pack(v):
    """MXFP4 bytes and scale bytes of v [..., m]."""
    r, e = _rounded(v)
    code = torch.bucketize(r, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)).to(torch.uint8)
    code = code.flatten(-2) | (torch.signbit(v).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _values(q, scales):
    """fp32 values of MXFP4 bytes q [..., m / 2] and scales [..., m / 32]."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=q.device)
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    v = grid[code.to(torch.int32)]
    p = (scales.to(torch.int32) << 23).view(torch.float32)     # 2^(byte - 127)
    return v.unflatten(-1, (-1, 32)).mul_(p.unsqueeze(-1)).flatten(-2)


def _plain_dispatch(case, s):
    counts, seg, dst = _layout(s["ids"], case["L"], case["align"])
    rows, k = s["rows"], case["k"]
    v = _quantised(s["x"].float()).to(torch.bfloat16)
    out = v.new_zeros(rows + 1, case["H"])
    to = torch.where(dst >= 0, dst, rows).long()
    out.index_copy_(0, to, v.repeat_interleave(k, 0))
    return {"rows": out[:rows], "src2dst": dst, "counts": counts}


def _grouped(a, w, counts, seg, most):
    """fp32 products of the rows a [R, K] in segments with w [L, N, K]; rows behind an expert's count are 0."""
    R = a.shape[0]
    at = (seg[:-1, None] + torch.arange(most, device=a.device)).clamp(max=R - 1)
    y = torch.bmm(w, a[at].transpose(1, 2).contiguous())       # [L, N, most]
    r = torch.arange(R, device=a.device)
    e = torch.searchsorted(seg[1:], r, right=True).clamp(max=w.shape[0] - 1)
    m = r - seg[e]
    got = y[e, :, m.clamp(min=0, max=most - 1)]
    return torch.where((m < counts[e]).unsqueeze(1), got, 0.0)


def _plain_product(case, s):
    a, w = _values(*s["a"]), _values(*s["w"])
    counts = s["counts"].long()
    if not case["masked"]:
        s["out"].copy_(_grouped(a, w, counts, s["seg"], s["most"]))
        return s["out"]
    y = torch.bmm(a[:, :s["most"]], w.transpose(1, 2).contiguous())
    live = torch.arange(s["most"], device=a.device) < counts[:, None]
    s["out"][:, :s["most"]] = torch.where(live.unsqueeze(-1), y, 0.0).to(torch.bfloat16)
    return s["out"]


def _swiglu(gu):
    g, u = gu.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def _plain_experts(case, s):
    T, k = case["T"], case["k"]
    counts, seg, dst = _layout(s["ids"], case["L"], case["align"])
    counts, valid = counts.long(), dst >= 0
    rows = s["rows"]
    a = s["x"].new_zeros(rows + 1, case["H"], dtype=torch.float32)
    a.index_copy_(0, torch.where(valid, dst, rows).long(), _quantised(s["x"].float()).repeat_interleave(k, 0))
    h = _swiglu(_grouped(a[:rows], _values(*s["w13"]), counts, seg, s["most"]))
    y = _grouped(_quantised(h), _values(*s["w2"]), counts, seg, s["most"])
    wt = torch.where(valid, s["weights"].reshape(-1), 0.0).unsqueeze(1)
    return (y[dst.clamp(min=0).long()] * wt).view(T, k, -1).sum(1).to(torch.bfloat16)


def _plain_layer(case, s):
    T, k, L = case["T"], case["k"], case["L"]
    ids = s["ids"].long()
    valid = (ids >= 0) & (ids < L)
    wt = torch.where(valid, s["weights"], 0.0)
    x = s["x"].float()
    four = case["weights"] == "mxfp4"
    if T * k <= L:                       # fewer slots than experts: the slots' own weights
        e = torch.where(valid, ids, 0).reshape(-1)
        w13 = _values(s["w13"][0][e], s["w13"][1][e]) if four else s["w13"][e].float()
        w2 = _values(s["w2"][0][e], s["w2"][1][e]) if four else s["w2"][e].float()
        h = _swiglu(torch.bmm(w13, x.repeat_interleave(k, 0).unsqueeze(2)).squeeze(2))
        y = torch.bmm(w2, h.unsqueeze(2)).squeeze(2)
        return (y * wt.reshape(-1, 1)).view(T, k, -1).sum(1).to(torch.bfloat16)
    w13 = _values(*s["w13"]) if four else s["w13"].float()
    w2 = _values(*s["w2"]) if four else s["w2"].float()
    # every token through every local expert, then the routed ones' weights
    gu = torch.matmul(w13.flatten(0, 1), x.t().contiguous()).view(L, -1, T).transpose(1, 2)
    h = _swiglu(gu).transpose(1, 2).contiguous()
    y = torch.bmm(w2, h)                                         # [L, H, T]
    per = torch.zeros(T, L + 1, device=x.device).scatter_add_(1, torch.where(valid, ids, L), wt)[:, :L]
    return (y * per.t().unsqueeze(1)).sum(0).t().contiguous().to(torch.bfloat16)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    T, E, L, k = case["T"], case["E"], case["L"], case["k"]
    R = T * k * L / E                                            # expected local slots
    U = T * (1 - math.prod((E - L - j) / (E - j) for j in range(k)))  # tokens with one
    active = L * (1 - (1 - k / E) ** T)                          # experts with one
    four = 17 / 32                                               # bytes of an MXFP4 element
    if case["kind"] == "dispatch":
        H = case["H"]
        return {"bytes": T * k * 4 + U * H * 2 + 2 * R * H * four + R * H * 2 + T * k * 4, "flops": 0}
    if case["kind"] == "product":
        K, N = case["K"], case["N"]
        return {"bytes": R * K * four + active * N * K * four + R * N * 2, "flops": 2 * R * K * N}
    H, I = case["H"], case["I"]
    each = 2 if case.get("weights") == "bf16" else four
    return {"bytes": T * k * 8 + U * H * 2 + active * 3 * I * H * each + T * H * 2, "flops": 6 * R * H * I}


def _exact_values(q, scales):
    lo, hi = (q & 15).long(), (q >> 4).long()
    v = torch.stack([lo, hi], dim=-1).reshape(*q.shape[:-1], -1, 32)
    mant, ex = (v & 1).double(), (v >> 1) & 3
    mag = torch.where(ex == 0, mant * 0.5, (1 + mant * 0.5) * torch.pow(2.0, (ex - 1).double()))
    mag = torch.where(v >= 8, -mag, mag)
    return (mag * torch.pow(2.0, scales.double() - 127).unsqueeze(-1)).reshape(*q.shape[:-1], -1)


def _exact_quantised(v):
    """MXFP4 values of v [rows, m] in 64 bits: the nearest grid value, halfway to the even code."""
    grid = torch.tensor(GRID, device=v.device, dtype=torch.float64)
    b = v.double().reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 6))
    e = torch.where(6 * torch.pow(2.0, e - 1) >= top, e - 1, e)
    e = torch.where(6 * torch.pow(2.0, e) < top, e + 1, e).clamp(min=-127)
    t = b.abs() / torch.pow(2.0, e)
    up = torch.bucketize(t, grid).clamp(max=7)
    lo = (up - 1).clamp(min=0)
    dl, du = t - grid[lo], grid[up] - t
    code = torch.where(dl < du, lo, torch.where(du < dl, up, torch.where(lo % 2 == 0, lo, up)))
    return (grid[code] * torch.pow(2.0, e) * torch.where(b < 0, -1.0, 1.0)).reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    kind, T, L, k = case["kind"], case["T"], case["L"], case["k"]
    if kind == "product":
        K, N = case["K"], case["N"]
        counts = s["counts"].tolist()
        q, sc = s["a"]
        first = [e * T for e in range(L)] if case["masked"] else s["seg"].tolist()
        q, sc = q.reshape(-1, K // 2), sc.reshape(-1, K // 32)
        y = torch.zeros(q.shape[0], N, device=DEV, dtype=torch.float64)
        for e in range(L):
            at = slice(first[e], first[e] + counts[e])
            if counts[e]:
                y[at] = _exact_values(q[at], sc[at]) @ _exact_values(s["w"][0][e], s["w"][1][e]).t()
        return y.view(L, T, N) if case["masked"] else y
    x, ids = s["x"], s["ids"].reshape(-1)
    token = torch.arange(T, device=DEV).repeat_interleave(k)
    slots = [(ids == e).nonzero().reshape(-1) for e in range(L)]
    if kind == "dispatch":
        v = _exact_quantised(x)
        out = torch.zeros(s["rows"], case["H"], device=DEV, dtype=torch.float64)
        begin, A = 0, case["align"]
        for e in range(L):
            out[begin:begin + len(slots[e])] = v[token[slots[e]]]
            begin += (len(slots[e]) + A - 1) // A * A
        return {"rows": out, "src2dst": None, "counts": None}
    w = s["weights"].reshape(-1).double()
    four = kind == "experts" or case["weights"] == "mxfp4"
    a = _exact_quantised(x) if kind == "experts" else x.double()
    out = torch.zeros(T, case["H"], device=DEV, dtype=torch.float64)
    for e in range(L):
        at = slots[e]
        if not len(at):
            continue
        w13 = _exact_values(s["w13"][0][e], s["w13"][1][e]) if four else s["w13"][e].double()
        w2 = _exact_values(s["w2"][0][e], s["w2"][1][e]) if four else s["w2"][e].double()
        gate, up = (a[token[at]] @ w13.t()).split(case["I"], 1)
        h = gate * torch.sigmoid(gate) * up
        h = _exact_quantised(h) if kind == "experts" else h
        out.index_add_(0, token[at], (h @ w2.t()) * w[at].unsqueeze(1))
    return out
