"""Cases for the operators whose weights depend on the activation row: expert
routing, packed products grouped by expert, the weighted sum of a token's
experts, and low-rank adapters beside a shared packed projection.

``run`` computes a case in plain torch operations (``own`` false) or through
this package's calls (``own`` true). Widths are those of the RWKV-7 layer sets
that the package benchmarks (2048/8192, 2560/10240, 4096); expert counts,
ranks and batch sizes are generic.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = {"w4g64": 64, "w8g16": 16, "w8g64": 64, "w6g16": 16}
RECORD = {"w4sb32": 144, "w5sb32": 176, "w6sb32": 208}
BITS = {"w4g64": 4, "w8g16": 8, "w8g64": 8, "w6g16": 6, "w4sb32": 4, "w5sb32": 5, "w6sb32": 6}
FORMATS = tuple(GROUP) + tuple(RECORD)


def listed():
    return [
        # one new token of one request: the router's latency
        {"name": "route one token", "op": "route", "T": 1, "E": 64, "k": 4, "dtype": "float32", "renorm": True},
        # a long prompt through a router with many experts, some of them masked
        {"name": "route prompt", "op": "route", "T": 8191, "E": 64, "k": 4, "dtype": "bfloat16", "renorm": True},
        # a decode batch's expert outputs joined
        {"name": "combine batch", "op": "combine", "T": 32, "k": 2, "N": 2048, "dtype": "bfloat16"},
        # a prompt's expert outputs joined: pure bandwidth
        {"name": "combine prompt", "op": "combine", "T": 8192, "k": 2, "N": 4096, "dtype": "bfloat16"},
        # one token at its two experts (channel-mix key width): the launch's latency and two matrices
        {"name": "experts one token", "op": "grouped", "fmt": "w4g64", "T": 1, "k": 2, "E": 16, "K": 2048, "N": 8192,
         "act": "relu2", "out": "bfloat16", "idle": 0, "tail": 0},
        # a decode batch whose rows reach nearly every expert: the whole weight stream
        {"name": "experts batch", "op": "grouped", "fmt": "w4g64", "T": 32, "k": 2, "E": 16, "K": 2048, "N": 8192,
         "act": "relu2", "out": "bfloat16", "idle": 0, "tail": 0},
        # the same batch size on the way down, 8-bit experts, long rows
        {"name": "experts batch int8 down", "op": "grouped", "fmt": "w8g16", "T": 24, "k": 2, "E": 8, "K": 8192,
         "N": 2048, "act": "none", "out": "bfloat16", "idle": 1, "tail": 0},
        # a short prompt, superblock weights, an odd width, experts without rows, padding rows behind the last group
        {"name": "experts ragged", "op": "grouped", "fmt": "w4sb32", "T": 333, "k": 1, "E": 8, "K": 2560, "N": 2501,
         "act": "none", "out": "float32", "idle": 3, "tail": 19},
        # a long prompt: the products are bound by arithmetic
        {"name": "experts prompt", "op": "grouped", "fmt": "w4g64", "T": 2048, "k": 2, "E": 8, "K": 2048, "N": 8192,
         "act": "relu2", "out": "bfloat16", "idle": 0, "tail": 0},
        # one request decoding with its adapter
        {"name": "adapter one token", "op": "lora", "fmt": "w4g64", "M": 1, "K": 2048, "N": 2048, "n": 8, "r": 16,
         "out": "float32", "ragged": False},
        # a decode batch, a different adapter on most rows, some rows without one
        {"name": "adapters batch", "op": "lora", "fmt": "w8g16", "M": 32, "K": 4096, "N": 4096, "n": 16, "r": 32,
         "out": "bfloat16", "ragged": False},
        # the largest activation block, many adapters of different ranks
        {"name": "adapters block", "op": "lora", "fmt": "w4sb32", "M": 128, "K": 2560, "N": 10240, "n": 24, "r": 64,
         "out": "bfloat16", "ragged": True},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("grouped", "grouped", "grouped", "lora", "lora", "route", "combine"))
    if op == "route":
        E = _logint(rng, 2, 256)
        return {"op": op, "T": _logint(rng, 1, 8192), "E": E, "k": rng.randint(1, min(8, E)),
                "dtype": rng.choice(("float32", "bfloat16")), "renorm": rng.random() < 0.5}
    if op == "combine":
        return {"op": op, "T": _logint(rng, 1, 6000), "k": rng.randint(1, 4), "N": _logint(rng, 256, 4096),
                "dtype": rng.choice(("float32", "bfloat16"))}
    fmt = rng.choice(FORMATS)
    unit = 256 if fmt in RECORD else 64
    K = unit * max(1, _logint(rng, 256, 8192) // unit)
    if op == "lora":
        N = _logint(rng, 200, 8192)
        return {"op": op, "fmt": fmt, "M": _logint(rng, 1, 128), "K": K, "N": N, "n": rng.randint(1, 24),
                "r": 8 * rng.randint(1, 8), "out": rng.choice(("float32", "bfloat16")), "ragged": rng.random() < 0.5}
    E = _logint(rng, 2, 32)
    N = min(_logint(rng, 200, 8192), (1 << 27) // (E * K))
    k = rng.randint(1, min(3, E))
    T = max(1, min(_logint(rng, 1, 2048), (1 << 35) // (K * N * k)))
    return {"op": op, "fmt": fmt, "T": T, "k": k, "E": E, "K": K, "N": N, "act": rng.choice(("none", "relu2")),
            "out": rng.choice(("float32", "bfloat16")), "idle": rng.randint(0, (E - k) // 2),
            "tail": rng.choice((0, 0, 5, 40))}


# ------------------------------------------------------------------ inputs --
def _dtype(name):
    return {"float32": torch.float32, "bfloat16": torch.bfloat16}[name]


def _planes(fmt, rows, K, g):
    """The code and scale planes of a packed matrix: codes spread as those of
    normally distributed weights, scales as of weights of deviation 0.02."""
    if fmt in RECORD:
        rec = torch.randint(0, 256, (rows, K // 256, RECORD[fmt]), generator=g, device=DEV, dtype=torch.uint8)
        step = 0.12 / (2 ** BITS[fmt] - 1) / 48
        head = torch.rand(rows, K // 256, 2, generator=g, device=DEV) * 0.4 + 0.8
        head = (head * torch.tensor([step, 0.06 / 48], device=DEV)).to(torch.float16)
        rec[..., :4] = head.view(torch.uint8)
        rec[..., 4:16] |= 0x82                       # the larger half of the 6-bit fields, mostly
        return rec.reshape(-1), None
    G, top = GROUP[fmt], 2 ** (BITS[fmt] - 1) - 1
    q = torch.randn(rows, K, generator=g, device=DEV, dtype=torch.float16).mul_(top / 2.5).round_().clamp_(-top, top)
    u = q.add_(top + 1).to(torch.uint8)
    del q
    if fmt == "w4g64":
        codes = u[:, 0::2] | (u[:, 1::2] << 4)
    elif fmt == "w6g16":
        c = u.view(rows, K // 64, 64)
        low = (c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)
        high = (c[..., 0::4] >> 4) | ((c[..., 1::4] >> 4) << 2) | ((c[..., 2::4] >> 4) << 4) | ((c[..., 3::4] >> 4) << 6)
        codes = torch.cat((low, high), -1)
    else:
        codes = u
    s = torch.rand(rows * (K // G), generator=g, device=DEV) * 0.4 + 0.8
    s = (s * (0.05 / top)).to(torch.float16).view(torch.uint8)
    pad = -s.numel() % 16
    return codes.reshape(-1), torch.cat((s, s.new_zeros(pad))) if pad else s


def _activations(rows, K, g):
    """bf16 rows with a few channels far above the others, as in the residual stream."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    x[:, 5::509] *= 12.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)
    s = {"case": c}
    if c["op"] == "route":
        l = torch.randn(c["T"], c["E"], generator=g, device=DEV) * 2
        gone = torch.rand(c["T"], c["E"], generator=g, device=DEV) < 0.05
        gone |= torch.rand(c["T"], 1, generator=g, device=DEV) < 0.01           # rows that a mask leaves empty
        s["logits"] = l.masked_fill(gone, -math.inf).to(_dtype(c["dtype"]))
        if own:
            from weight_only_quantized_rq_b200 import TopkRouter
            s["router"] = TopkRouter(c["E"], c["k"], renorm=c["renorm"])
    elif c["op"] == "combine":
        T, k, N = c["T"], c["k"], c["N"]
        s["y"] = torch.randn(T * k, N, generator=g, device=DEV).to(_dtype(c["dtype"]))
        s["ids"] = torch.randint(0, 16, (T, k), generator=g, device=DEV, dtype=torch.int32)
        gone = torch.rand(T, k, generator=g, device=DEV) < 0.03
        s["ids"][gone] = -1
        s["y"][gone.view(-1)] = math.nan                                        # a slot without an expert is never written
        s["weights"] = torch.rand(T, k, generator=g, device=DEV).masked_fill(gone, 0.0)
    elif c["op"] == "grouped":
        T, k, E, K, N = c["T"], c["k"], c["E"], c["K"], c["N"]
        h = torch.Generator().manual_seed(seed * 104729 + 7)
        pull = torch.randn(E, generator=h) * 0.7                                # some experts draw more tokens
        pull[torch.randperm(E, generator=h)[:c["idle"]]] = -math.inf            # and some none
        noise = -torch.log(-torch.log(torch.rand(T, E, generator=h).clamp(1e-7, 1 - 1e-7)))
        ids = (pull + noise).topk(k, -1).indices.reshape(-1)
        order = ids.argsort(stable=True)
        counts = torch.bincount(ids, minlength=E)
        s["cap"] = max(1, int(counts.max()))
        R = T * k + c["tail"]
        s["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64), counts.cumsum(0))).to(torch.int32).to(DEV)
        rows = torch.full((R,), -1, dtype=torch.int32)
        rows[:T * k] = (order // k).to(torch.int32)
        s["in_rows"] = rows.to(DEV)
        s["x"] = _activations(T, K, g)
        s["codes"], s["scales"] = _planes(c["fmt"], E * N, K, g)
        s["y"] = torch.zeros(R, N, dtype=_dtype(c["out"]), device=DEV)
        if own:
            from weight_only_quantized_rq_b200 import GroupedExperts, Packed, fmt_id
            s["experts"] = GroupedExperts(Packed(fmt_id(c["fmt"]), K, E * N, s["codes"], s["scales"]), E, max_rows=R)
    else:
        M, K, N, n, r = c["M"], c["K"], c["N"], c["n"], c["r"]
        s["x"] = _activations(M, K, g)
        s["codes"], s["scales"] = _planes(c["fmt"], N, K, g)
        s["A"] = (torch.randn(n, r, K, generator=g, device=DEV) / math.sqrt(K)).to(torch.bfloat16)
        s["B"] = (torch.randn(n, N, r, generator=g, device=DEV) * (0.3 / math.sqrt(r))).to(torch.bfloat16)
        s["alpha"] = torch.rand(n, generator=g, device=DEV) + 0.5
        if c["ragged"]:
            s["ranks"] = 8 * torch.randint(1, r // 8 + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
        else:
            s["ranks"] = torch.full((n,), r, dtype=torch.int32, device=DEV)
        a = torch.randint(0, n, (M,), generator=g, device=DEV, dtype=torch.int32)
        if M > 1:
            a[torch.rand(M, generator=g, device=DEV) < 0.1] = -1
        s["adapter"] = a
        if own:
            from weight_only_quantized_rq_b200 import LoraProjection, Packed, fmt_id
            s["projection"] = LoraProjection(Packed(fmt_id(c["fmt"]), K, N, s["codes"], s["scales"]), s["A"], s["B"],
                                             s["alpha"], s["ranks"], max_rows=M)
    return s


# -------------------------------------------------------------- plain form --
def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _dequant(fmt, codes, scales, rows, K):
    if fmt in RECORD:
        rec = codes.view(rows, K // 256, RECORD[fmt])
        head = rec[..., :4].contiguous().view(torch.float16).float()
        by = torch.arange(6, device=codes.device) * 8
        at = torch.arange(8, device=codes.device) * 6
        sc = ((rec[..., 4:10].long() << by).sum(-1, keepdim=True) >> at) & 63
        mn = ((rec[..., 10:16].long() << by).sum(-1, keepdim=True) >> at) & 63
        q = _nibbles(rec[..., 16:144])
        if fmt == "w5sb32":
            high = (rec[..., 144:].unsqueeze(-1) >> torch.arange(8, device=codes.device, dtype=torch.uint8)) & 1
            q = q | (high.flatten(-2) << 4)
        elif fmt == "w6sb32":
            high = (rec[..., 144:].unsqueeze(-1) >> (2 * torch.arange(4, device=codes.device, dtype=torch.uint8))) & 3
            q = q | (high.flatten(-2) << 4)
        S, Mn = head[..., :1] * sc, head[..., 1:] * mn
        return (q.view(rows, K // 256, 8, 32) * S.unsqueeze(-1) - Mn.unsqueeze(-1)).view(rows, K)
    G = GROUP[fmt]
    if fmt == "w4g64":
        q = _nibbles(codes.view(rows, K // 2))
    elif fmt == "w6g16":
        c = codes.view(rows, K // 64, 48)
        high = (c[..., 32:].unsqueeze(-1) >> (2 * torch.arange(4, device=codes.device, dtype=torch.uint8))) & 3
        q = _nibbles(c[..., :32]) | (high.flatten(-2) << 4)
    else:
        q = codes
    s = scales[:rows * (K // G) * 2].view(torch.float16).float()
    return ((q.reshape(rows, K // G, G).float() - 2 ** (BITS[fmt] - 1)) * s.view(rows, K // G, 1)).view(rows, K)


def _plain_route(s):
    c, E = s["case"], s["case"]["E"]
    l = s["logits"].float()
    T, k = l.shape[0], c["k"]
    dead = l == -math.inf
    best, ids = torch.sort(l, dim=-1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k].to(torch.int32)
    top = best[:, :1].clamp(min=-3e38)
    w = torch.exp(best - top)
    w = w / (w.sum(-1, keepdim=True) if c["renorm"] else torch.exp(l - top).sum(-1, keepdim=True))
    none = best == -math.inf
    w = w.masked_fill(none, 0.0)
    ids = ids.masked_fill(none, -1)
    flat = ids.view(-1)
    key, order = torch.sort(torch.where(flat < 0, E, flat), stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=key.device, dtype=key.dtype)).to(torch.int32)
    slots = torch.where(key < E, order, -1).to(torch.int32)
    return ids, w, offsets, torch.where(key < E, order // k, -1).to(torch.int32), slots


def _plain_combine(s):
    c = s["case"]
    y = s["y"].view(c["T"], c["k"], c["N"]).float()
    y = torch.where((s["ids"] >= 0).unsqueeze(-1), y * s["weights"].unsqueeze(-1), 0.0)
    return y.sum(1).to(s["y"].dtype)


def _plain_grouped(s):
    c = s["case"]
    E, K, N, R = c["E"], c["K"], c["N"], s["y"].shape[0]
    W = _dequant(c["fmt"], s["codes"], s["scales"], E * N, K).view(E, N, K)
    off = s["offsets"].long()
    i = torch.arange(R, device=off.device)
    live = i < off[-1]
    e = torch.searchsorted(off[1:], i, right=True).clamp(max=E - 1)
    at = torch.where(live, e * s["cap"] + i - off[e], E * s["cap"])           # a row of its own for the tail
    P = torch.zeros(E * s["cap"] + 1, K, device=off.device)
    P[at] = s["x"][s["in_rows"].long().clamp(min=0)].float()
    Y = torch.bmm(P[:-1].view(E, s["cap"], K), W.transpose(1, 2)).view(-1, N)
    y = Y[at.clamp(max=E * s["cap"] - 1)]
    if c["act"] == "relu2":
        y = y.clamp(min=0).square()
    return torch.where(live.unsqueeze(-1), y.to(s["y"].dtype), s["y"])


def _plain_lora(s):
    c = s["case"]
    x = s["x"].float()
    y = x @ _dequant(c["fmt"], s["codes"], s["scales"], c["N"], c["K"]).t()
    a = s["adapter"].long()
    at = a.clamp(min=0)
    t = torch.bmm(s["A"][at].float(), x.unsqueeze(-1)).squeeze(-1)
    t = t * (torch.arange(c["r"], device=t.device) < s["ranks"][at].unsqueeze(-1))
    t = t * torch.where(a >= 0, s["alpha"][at], 0.0).unsqueeze(-1)
    y = y + torch.bmm(s["B"][at].float(), t.unsqueeze(-1)).squeeze(-1)
    return y.to(_dtype(c["out"]))


def run(state):
    c = state["case"]
    if own:
        if c["op"] == "route":
            r = state["router"](state["logits"])
            return r.ids, r.weights, r.offsets, r.in_rows, r.slots
        if c["op"] == "combine":
            from weight_only_quantized_rq_b200 import rq_route_combine
            return rq_route_combine(state["y"], state["ids"], state["weights"])
        if c["op"] == "grouped":
            return state["experts"](state["x"], state["offsets"], in_rows=state["in_rows"], y=state["y"],
                                    act=None if c["act"] == "none" else c["act"])
        return state["projection"](state["x"], state["adapter"], out_dtype=_dtype(c["out"]))
    return {"route": _plain_route, "combine": _plain_combine, "grouped": _plain_grouped, "lora": _plain_lora}[c["op"]](state)


def _plane_bytes(fmt, rows, K):
    if fmt in RECORD:
        return rows * (K // 256) * RECORD[fmt]
    return rows * K * BITS[fmt] // 8 + rows * (K // GROUP[fmt]) * 2


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": c["T"] * c["E"] * size + 16 * c["T"] * c["k"] + 4 * (c["E"] + 1), "flops": 0}
    if c["op"] == "combine":
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": c["T"] * (c["k"] + 1) * c["N"] * size + 8 * c["T"] * c["k"], "flops": 2 * c["T"] * c["k"] * c["N"]}
    size = 4 if c["out"] == "float32" else 2
    if c["op"] == "grouped":
        R, live = c["T"] * c["k"], c["E"] - c["idle"]
        used = live * (1 - (1 - c["k"] / live) ** c["T"])                       # experts that rows reach
        return {"bytes": int(used * _plane_bytes(c["fmt"], c["N"], c["K"])) + 2 * c["T"] * c["K"] + size * R * c["N"] + 4 * R,
                "flops": 2 * R * c["K"] * c["N"]}
    used = c["n"] * (1 - (1 - 1 / c["n"]) ** c["M"])
    rank = c["r"] * (0.55 if c["ragged"] else 1)
    return {"bytes": int(_plane_bytes(c["fmt"], c["N"], c["K"]) + 2 * used * rank * (c["K"] + c["N"])) + 2 * c["M"] * c["K"] +
            size * c["M"] * c["N"], "flops": int(2 * c["M"] * (c["K"] * c["N"] + rank * (c["K"] + c["N"])))}


# ------------------------------------------------------------------- exact --
def _field(bits, width):
    """Unsigned values of consecutive `width`-bit fields of a bit string (last axis, lowest bit first)."""
    w = (2.0 ** torch.arange(width, device=bits.device)).double()
    return bits.reshape(*bits.shape[:-1], -1, width).double() @ w


def _bits(b):
    return (b.unsqueeze(-1).to(torch.int16).bitwise_and(2 ** torch.arange(8, device=b.device, dtype=torch.int16)) > 0).flatten(-2)


def _weights64(fmt, codes, scales, row0, rows, K):
    """Rows row0 .. row0 + rows - 1 of w_hat in 64 bits, read from the layout's bit strings."""
    if fmt in RECORD:
        n, sz = K // 256, RECORD[fmt]
        rec = codes[row0 * n * sz:(row0 + rows) * n * sz].view(rows, n, sz)
        d = rec[..., 0:2].contiguous().view(torch.float16).double()
        m = rec[..., 2:4].contiguous().view(torch.float16).double()
        f = _field(_bits(rec[..., 4:16]), 6)
        q = _field(_bits(rec[..., 16:144]), 4)
        if sz > 144:
            q = q + 16 * _field(_bits(rec[..., 144:]), BITS[fmt] - 4)
        return (q.view(rows, n, 8, 32) * (d * f[..., :8]).unsqueeze(-1) - (m * f[..., 8:]).unsqueeze(-1)).view(rows, K)
    G, b = GROUP[fmt], BITS[fmt]
    per = K * b // 8
    c = codes[row0 * per:(row0 + rows) * per].view(rows, per)
    if fmt == "w6g16":
        c = c.view(rows, K // 64, 48)
        q = (_field(_bits(c[..., :32]), 4) + 16 * _field(_bits(c[..., 32:]), 2)).view(rows, K)
    else:
        q = _field(_bits(c), b)
    sc = scales.view(torch.float16)[row0 * (K // G):(row0 + rows) * (K // G)].double()
    return ((q - 2 ** (b - 1)).view(rows, K // G, G) * sc.view(rows, K // G, 1)).view(rows, K)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "route":
        p = torch.softmax(s["logits"].double().nan_to_num(neginf=-1e300), -1)
        p = p.masked_fill(s["logits"] == -math.inf, 0.0)
        w = p.sort(-1, descending=True).values[:, :c["k"]]
        if c["renorm"]:
            w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
        return None, w, None, None, None
    if c["op"] == "combine":
        out = torch.zeros(c["T"], c["N"], dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            out += s["y"][j::c["k"]].double().nan_to_num(0.0) * s["weights"][:, j:j + 1].double()
        return out
    if c["op"] == "grouped":
        y = s["y"].double()
        off = s["offsets"].tolist()
        for e in range(c["E"]):
            if off[e + 1] > off[e]:
                v = s["x"][s["in_rows"][off[e]:off[e + 1]].long()].double()
                for n0 in range(0, c["N"], 1024):
                    n1 = min(c["N"], n0 + 1024)
                    v_w = v @ _weights64(c["fmt"], s["codes"], s["scales"], e * c["N"] + n0, n1 - n0, c["K"]).t()
                    y[off[e]:off[e + 1], n0:n1] = v_w.relu() ** 2 if c["act"] == "relu2" else v_w
        return y
    x = s["x"].double()
    y = torch.cat([x @ _weights64(c["fmt"], s["codes"], s["scales"], n0, min(1024, c["N"] - n0), c["K"]).t()
                   for n0 in range(0, c["N"], 1024)], 1)
    for m, a in enumerate(s["adapter"].tolist()):
        if a >= 0:
            r = int(s["ranks"][a])
            t = s["A"][a, :r].double() @ x[m]
            y[m] += s["alpha"][a].double() * (s["B"][a, :, :r].double() @ t)
    return y
