"""Measured cases of the operators on 4-bit weights with group scales.

Three operators of a layer whose weights are held as 4-bit codes with one scale (and, where asked
for, one zero point) per group of input columns:

  quantize  W -> codes, scales, zero points, and the values they stand for read back
  matmul    Y = X W^T for one token up to a long prompt
  moe       a mixture-of-experts layer (router, gate/up, down) for a few tokens

``run`` computes them in plain torch operations, or through the library where ``own`` is true.

Format: code of column k is nibble k % 8 (lowest first) of 32-bit word k // 8; a row has
4 ceil(n / 32) words; W^ = scale (code - zero), zero = 8 where there is no array of zero points.
"""
import math

import torch

own = False
if own:
    import rank_binary_factorization_b200  # noqa: F401


def listed():
    return [
        # the small planted matrix of the tests, FP32, finest groups: latency of a quantiser call
        dict(name="quantize 256x512 f32 g32 zeros", op="quantize", m=256, n=512, bf16=False,
             group=32, zeros=True, grid=1, weighted=False),
        # a square attention projection with the calibrated clipping search
        dict(name="quantize 4096x4096 bf16 g128 grid16", op="quantize", m=4096, n=4096, bf16=True,
             group=128, zeros=False, grid=16, weighted=True),
        # the largest projection of the configurations, rounding to nearest only
        dict(name="quantize 28672x8192 bf16 g64 zeros", op="quantize", m=28672, n=8192, bf16=True,
             group=64, zeros=True, grid=1, weighted=False),
        # decoding one token: attention projection
        dict(name="matmul 4096x4096 bf16 B1 g128", op="matmul", m=4096, n=4096, bf16=True,
             group=128, zeros=False, batch=1),
        # decoding one token: the widest projection of the 4096-wide block
        dict(name="matmul 11008x4096 bf16 B1 g64 zeros", op="matmul", m=11008, n=4096, bf16=True,
             group=64, zeros=True, batch=1),
        # odd sizes, FP32 activations, three requests decoding together
        dict(name="matmul 1000x777 f32 B3 g32 zeros", op="matmul", m=1000, n=777, bf16=False,
             group=32, zeros=True, batch=3),
        # sixteen requests decoding together through the largest projection
        dict(name="matmul 28672x8192 bf16 B16 g128", op="matmul", m=28672, n=8192, bf16=True,
             group=128, zeros=False, batch=16),
        # a short prompt, FP32 activations, long sums
        dict(name="matmul 4096x11008 f32 B100 g128 zeros", op="matmul", m=4096, n=11008, bf16=False,
             group=128, zeros=True, batch=100),
        # one calibration sequence of 2048 tokens
        dict(name="matmul 11008x4096 bf16 B2048 g128", op="matmul", m=11008, n=4096, bf16=True,
             group=128, zeros=False, batch=2048),
        # one token through many small experts
        dict(name="moe B1 E64 k6 2048x1408 bf16 g128", op="moe", batch=1, experts=64, top_k=6,
             d=2048, f=1408, bf16=True, group=128, zeros=False, renormalise=True),
        # several requests: most experts are used, by one or two tokens each
        dict(name="moe B8 E64 k8 4096x1024 bf16 g64 zeros", op="moe", batch=8, experts=64, top_k=8,
             d=4096, f=1024, bf16=True, group=64, zeros=True, renormalise=True),
        # few large experts, each used by several tokens, FP32 activations
        dict(name="moe B16 E8 k2 4096x11008 f32 g128", op="moe", batch=16, experts=8, top_k=2,
             d=4096, f=11008, bf16=False, group=128, zeros=False, renormalise=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _size(rng, lo, hi):
    """A size between lo and hi: half the time a multiple of 64, else any number."""
    v = _spread(rng, lo, hi)
    return max(lo, v // 64 * 64) if rng.random() < 0.5 and v >= 64 else v


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "moe"])
    case = dict(op=op, bf16=rng.random() < 0.6, group=rng.choice([32, 64, 128]),
                zeros=rng.random() < 0.5)
    if op == "quantize":
        grid = rng.choice([1, 1, 4, 16])
        n = _size(rng, 100, 8192)
        m = _size(rng, 64, min(28672, 28672 * 8192 // (n * grid)))
        case.update(m=m, n=n, grid=grid, weighted=rng.random() < 0.5)
    elif op == "matmul":
        m, n = _size(rng, 256, 28672), _size(rng, 256, 8192)
        case.update(m=m, n=n, batch=_spread(rng, 1, min(2048, 11008 * 4096 * 2048 // (m * n))))
    else:
        experts = _spread(rng, 4, 64)
        d = _size(rng, 256, 4096)
        f = _size(rng, 128, min(11008, 8 * 4096 * 11008 // (experts * d)))
        case.update(experts=experts, top_k=rng.randint(1, min(8, experts)), d=d, f=f,
                    batch=_spread(rng, 1, 16), renormalise=rng.random() < 0.5)
    return case


# ---- inputs ---------------------------------------------------------------------------
def _codes(rows, n, group, zeros, gen):
    """Packed codes, scales and zero points as rounding normal weights of std 0.02 gives them."""
    ld, ng = 4 * -(-n // 32), -(-n // group)
    nib = torch.empty(rows, 8 * ld, dtype=torch.float16, device="cuda").normal_(8, 2.4, generator=gen)
    nib = nib.round_().clamp_(0, 15).to(torch.uint8)
    packed = (nib[:, 0::2] | (nib[:, 1::2] << 4)).view(torch.int32)
    s = torch.empty(rows, ng, device="cuda").normal_(math.log(0.0083), 0.2, generator=gen).exp_()
    z = None
    if zeros:
        z = torch.empty(rows, ng, device="cuda").normal_(7.5, 1, generator=gen).round_().clamp_(0, 15)
        z = z.to(torch.uint8)
    return packed, s.to(torch.bfloat16), z


def _acts(rows, n, bf16, gen):
    """Activations with log-normal channel scales."""
    x = torch.randn(rows, n, device="cuda", generator=gen)
    x *= torch.randn(n, device="cuda", generator=gen).mul_(0.5).exp_()
    return x.to(torch.bfloat16) if bf16 else x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    if case["op"] == "quantize":
        m, n = case["m"], case["n"]
        W = torch.empty(m, n, device="cuda").normal_(0, 0.02, generator=gen)
        wide = torch.randperm(n, device="cuda", generator=gen)[:max(1, n // 100)]
        W[:, wide] *= 10
        st["W"] = W.to(torch.bfloat16) if case["bf16"] else W
        d = torch.randn(n, device="cuda", generator=gen).exp_()
        st["d_in"] = d if case["weighted"] else None
    elif case["op"] == "matmul":
        st["w"] = _codes(case["m"], case["n"], case["group"], case["zeros"], gen)
        st["X"] = _acts(case["batch"], case["n"], case["bf16"], gen)
    else:
        E, d, f, g = case["experts"], case["d"], case["f"], case["group"]

        def stacked(rows, n):
            return tuple(None if t is None else t.view(E, rows, -1)
                         for t in _codes(E * rows, n, g, case["zeros"], gen))

        st["gate_up"], st["down"] = stacked(2 * f, d), stacked(d, f)
        st["X"] = _acts(case["batch"], d, case["bf16"], gen)
        R = torch.randn(E, d, device="cuda", generator=gen) / math.sqrt(d)
        st["router"] = R.to(st["X"].dtype)
    return st


# ---- plain forms ----------------------------------------------------------------------
def _grouped(v, group, n):
    """One value per group to one per column."""
    return v.repeat_interleave(group, dim=-1)[..., :n]


def _values(w, group, n):
    """W^ = scale (code - zero) in FP32, of packed words (..., rows, ld)."""
    packed, scales, zeros = w
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device=packed.device)
    codes = ((packed.unsqueeze(-1) >> shifts) & 15).flatten(-2)[..., :n].float()
    z = 8.0 if zeros is None else _grouped(zeros.float(), group, n)
    return (codes - z) * _grouped(scales.float(), group, n)


def _plain_quantize(st):
    m, n, g, grid = st["m"], st["n"], st["group"], st["grid"]
    ng = -(-n // g)
    pad = ng * g - n
    w = torch.nn.functional.pad(st["W"].double(), (0, pad)).view(m, ng, g)
    d = torch.ones(n, device=w.device) if st["d_in"] is None else st["d_in"]
    d = torch.nn.functional.pad(d.double(), (0, pad)).view(ng, g)
    best = None
    for c in range(grid):      # the candidates of the clipping search
        alpha = 1 - c / (2 * grid)
        if st["zeros"]:
            lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
            s = (alpha * (hi - lo) / 15).float().to(torch.bfloat16)
            z = torch.where(s > 0, (-alpha * lo / s.double()).round().clamp(0, 15), 0.0)
        else:
            s = (alpha * w.abs().amax(-1) / 7).float().to(torch.bfloat16)
            z = torch.full_like(s, 8.0, dtype=torch.float64)
        sd = s.double().unsqueeze(-1)
        q = torch.where(sd > 0, (w / sd).round(), 0.0) + z.unsqueeze(-1)
        v = (q.clamp(0, 15) - z.unsqueeze(-1)) * sd
        err = ((w - v) * d).square().sum(-1)
        if best is None:
            best = (err, v, s, z)
        else:
            less = err < best[0]
            best = (torch.where(less, err, best[0]), torch.where(less.unsqueeze(-1), v, best[1]),
                    torch.where(less, s, best[2]), torch.where(less, z, best[3]))
    out = {"values": best[1].reshape(m, ng * g)[:, :n].to(st["W"].dtype), "scales": best[2]}
    if st["zeros"]:
        out["zeros"] = best[3].float()
    return out


def _plain_moe(st):
    X, k, E = st["X"], st["top_k"], st["experts"]
    d, f, g, B = st["d"], st["f"], st["group"], st["batch"]
    logits = X.double() @ st["router"].double().T
    top, order = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids = order[:, :k]
    over = top[:, :k] if st["renormalise"] else logits
    p = torch.exp(top[:, :k] - torch.logsumexp(over, -1, keepdim=True)).float()
    # the experts to compute: one per (token, choice), or all where that is fewer
    if B * k < E:
        sel, at = ids.reshape(-1), torch.arange(B * k, device=X.device).view(B, k)
    else:
        sel, at = torch.arange(E, device=X.device), ids
    pick = lambda w: tuple(None if t is None else t[sel] for t in w)  # noqa: E731
    gu = X.float() @ _values(pick(st["gate_up"]), g, d).transpose(1, 2)       # (S, B, 2f)
    gate, up = gu[..., :f], gu[..., f:]
    h = gate / (1 + torch.exp(-gate)) * up
    o = h @ _values(pick(st["down"]), g, f).transpose(1, 2)                   # (S, B, d)
    rows = torch.arange(B, device=X.device).unsqueeze(1)
    y = (o[at, rows] * p.unsqueeze(-1)).sum(1)
    return {"Y": y, "ids": ids.to(torch.int32), "weights": p}


def run(state):
    st = state
    if st["op"] == "quantize":
        if own:
            import rank_binary_factorization_b200 as nq
            q = nq.nq_w4_quantize(st["W"], group=st["group"], d_in=st["d_in"],
                                  symmetric=not st["zeros"], grid=st["grid"])
            v = nq.nq_w4_dequantize(q["packed"], q["scales"], st["n"], group=st["group"],
                                    zeros=q["zeros"], dtype=st["W"].dtype)
            out = {"values": v, "scales": q["scales"]}
            if st["zeros"]:
                out["zeros"] = q["zeros"].float()
            return out
        return _plain_quantize(st)
    if st["op"] == "matmul":
        packed, scales, zeros = st["w"]
        if own:
            import rank_binary_factorization_b200 as nq
            return nq.nq_w4_matmul(packed, scales, st["X"], group=st["group"], zeros=zeros)
        return st["X"].float() @ _values(st["w"], st["group"], st["n"]).T
    if own:
        import rank_binary_factorization_b200 as nq
        (gu, gu_s, gu_z), (dn, dn_s, dn_z) = st["gate_up"], st["down"]
        y, ids, p = nq.nq_moe_w4(st["X"], st["router"], gu, gu_s, dn, dn_s, st["top_k"],
                                 group=st["group"], gate_up_zeros=gu_z, down_zeros=dn_z,
                                 renormalise=st["renormalise"], want_routing=True)
        return {"Y": y, "ids": ids, "weights": p}
    return _plain_moe(st)


# ---- work -----------------------------------------------------------------------------
def _packed_bytes(rows, n, group, zeros):
    return rows * (16 * -(-n // 32) + -(-n // group) * (3 if zeros else 2))


def work(case):
    e = 2 if case["bf16"] else 4
    if case["op"] == "quantize":
        m, n = case["m"], case["n"]
        packed = _packed_bytes(m, n, case["group"], case["zeros"])
        # weights read, codes written, codes read back, values written
        return {"bytes": 2 * m * n * e + 2 * packed + (4 * n if case["weighted"] else 0),
                "flops": 8 * m * n * case["grid"]}
    if case["op"] == "matmul":
        m, n, B = case["m"], case["n"], case["batch"]
        return {"bytes": _packed_bytes(m, n, case["group"], case["zeros"]) + B * (n * e + 4 * m),
                "flops": 2 * B * m * n}
    E, k, d, f, B = case["experts"], case["top_k"], case["d"], case["f"], case["batch"]
    used = E * (1 - (1 - k / E) ** B)      # expected number of experts that some token chose
    per = (_packed_bytes(2 * f, d, case["group"], case["zeros"]) +
           _packed_bytes(d, f, case["group"], case["zeros"]))
    return {"bytes": used * per + E * d * e + B * d * (e + 4) + B * k * 8,
            "flops": 6 * B * k * d * f + 2 * B * E * d}


# ---- the definition in 64 bits ----------------------------------------------------------
def _exact_values(w, group, n):
    """Row-major float64 W^ of packed words (rows, ld), from the bytes of the words."""
    packed, scales, zeros = w
    b = packed.contiguous().view(torch.uint8).long()
    q = torch.stack((b % 16, b // 16), -1).reshape(b.shape[0], -1)[:, :n].double()
    col = torch.arange(n, device=b.device) // group
    q -= 8 if zeros is None else zeros.double()[:, col]
    return q.mul_(scales.double()[:, col])


def exact(case, seed):
    st = prepare(case, seed)
    g = case["group"]
    if case["op"] == "matmul":
        return _exact_values(st["w"], g, case["n"]).matmul(st["X"].double().T).T.contiguous()
    if case["op"] == "quantize":
        m, n, grid = case["m"], case["n"], case["grid"]
        values = torch.empty(m, n, dtype=torch.float64, device="cuda")
        scales = torch.empty(m, -(-n // g), dtype=torch.float64, device="cuda")
        zeros = torch.empty_like(scales)
        for j, a in enumerate(range(0, n, g)):
            w = st["W"][:, a:a + g].double()
            wt = 1.0 if st["d_in"] is None else st["d_in"][a:a + g].double() ** 2
            errs, vals, ss, zs = [], [], [], []
            for c in range(grid):
                keep = (2 * grid - c) / (2 * grid)
                if case["zeros"]:
                    lo = torch.minimum(w.min(1).values, torch.zeros((), device="cuda", dtype=w.dtype))
                    hi = torch.maximum(w.max(1).values, torch.zeros((), device="cuda", dtype=w.dtype))
                    s = (keep * (hi - lo) / 15).float().bfloat16().double()[:, None]
                    z = torch.clamp(torch.round(-keep * lo[:, None] / s), 0, 15)
                else:
                    s = (keep * w.abs().max(1).values / 7).float().bfloat16().double()[:, None]
                    z = torch.tensor(8.0, device="cuda", dtype=w.dtype)
                low, high = (0 - z) * s, (15 - z) * s
                v = torch.minimum(torch.maximum(torch.round(w / s) * s, low), high)
                errs.append((wt * (w - v) ** 2).sum(1))
                vals.append(v)
                ss.append(s[:, 0])
                zs.append(z.expand_as(s)[:, 0])
            pick = torch.stack(errs).min(0).indices       # no ties among normal weights
            rows = torch.arange(m, device="cuda")
            values[:, a:a + g] = torch.stack(vals)[pick, rows]
            scales[:, j] = torch.stack(ss)[pick, rows]
            zeros[:, j] = torch.stack(zs)[pick, rows]
        out = {"values": values, "scales": scales}
        if case["zeros"]:
            out["zeros"] = zeros
        return out
    B, k, f, d = case["batch"], case["top_k"], case["f"], case["d"]
    X = st["X"].double()
    logits = torch.stack([(X * r).sum(1) for r in st["router"].double()], 1).tolist()
    y = torch.zeros(B, d, dtype=torch.float64, device="cuda")
    ids, weights, users = [], [], {}
    for b, row in enumerate(logits):
        chosen = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        total = sum(math.exp(row[e] - max(row)) for e in (chosen if case["renormalise"] else range(len(row))))
        ids.append(chosen)
        weights.append([math.exp(row[e] - max(row)) / total for e in chosen])
        for e, p in zip(chosen, weights[-1]):
            users.setdefault(e, []).append((b, p))
    for e, pairs in users.items():
        part = lambda w: tuple(None if t is None else t[e] for t in w)  # noqa: E731
        x = X[[b for b, _ in pairs]]
        gu = x @ _exact_values(part(st["gate_up"]), g, d).T
        h = gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:]
        o = h @ _exact_values(part(st["down"]), g, f).T
        for (b, p), v in zip(pairs, o):
            y[b] += p * v
    return {"Y": y, "ids": torch.tensor(ids, dtype=torch.int32, device="cuda"),
            "weights": torch.tensor(weights, dtype=torch.float64, device="cuda")}
