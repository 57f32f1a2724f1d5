"""The operators around the experts of a mixture-of-experts layer, as cases to measure.

Three groups, beside the routing, align and forward entry points of the library:

  permute / permute_backward / unpermute / unpermute_backward
      tokens copied into expert order, and the experts' rows added back into tokens with
      the routing weights, each with its gradient;
  route_backward
      the gradient of the renormalised softmax top-k with respect to the router logits;
  lora / lora_backward
      low-rank adapters of many requests beside one shared projection:
      y = base + scale[g] * (x A[g]^T) B[g]^T with g the adapter of each row.

Shapes: the Qwen-shaped layer (E = 128, H = 2048, I = 768, k = 8) and the GLM-class layer
(E = 256, H = 6144, I = 2048, k = 8) of this repository's synthetic workloads, and odd
sizes around them. With `own` false, `run` computes each operator from elementary torch
operations in fp32; with `own` true it calls the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
# up to this many rows the plain adapters gather each row's own matrices; beyond it they
# multiply by every adapter at once and mask (memory M * r * K against M * G * r)
GATHER_ROWS = 64


def _layer(name, op, M, k, E, H, dtype="bf16", local=0, skew=0.0):
    """A case of the permutation group: M tokens of H values, k experts of E each; `local`:
    how many of the experts this process holds (0: all; slots of the others are dropped);
    `skew`: standard deviation of a per-expert bias on the router logits."""
    return dict(name=name, op=op, M=M, k=k, E=E, H=H, dtype=dtype, local=local, skew=skew)


def _lora(name, op, M, G, K, N, r, none=0.0, skew=0.0):
    """A case of the adapters: M rows, G adapters of rank r beside a projection K -> N;
    `none`: the share of rows without an adapter; `skew`: how uneven the adapters' use is."""
    return dict(name=name, op=op, M=M, G=G, K=K, N=N, r=r, none=none, skew=skew)


def listed():
    return [
        # one new token through the Qwen-shaped layer: its 8 slots in expert order
        _layer("permute_qwen_m1", "permute", 1, 8, 128, 2048),
        # a prefill chunk of the GLM-class layer with uneven expert load
        _layer("permute_glm_m4096", "permute", 4096, 8, 256, 6144, skew=1.0),
        # the same step's gradient in a training run that keeps fp32 rows, odd sizes
        _layer("permute_bwd_odd_m1021", "permute_backward", 1021, 6, 61, 2049, "fp32"),
        # a decode batch of the GLM-class layer: eight tokens put back together
        _layer("unpermute_glm_m8", "unpermute", 8, 8, 256, 6144),
        # the prefill chunk's combine
        _layer("unpermute_glm_m4096", "unpermute", 4096, 8, 256, 6144, skew=1.0),
        # gradient of the combine, one process's share of the experts (a quarter), fp16 rows
        _layer("unpermute_bwd_share_m4096", "unpermute_backward", 4096, 8, 256, 6144, "fp16", local=64),
        # router gradient of a small batch and of a long packed training sequence
        _layer("route_bwd_qwen_m8", "route_backward", 8, 8, 128, 2048),
        _layer("route_bwd_glm_m16384", "route_backward", 16384, 8, 256, 6144),
        # one request's token beside the Qwen-shaped up projection, and a decode batch of 64
        # requests that use 48 adapters beside the GLM-class one
        _lora("lora_qwen_m1", "lora", 1, 16, 2048, 1536, 16),
        _lora("lora_glm_m64", "lora", 64, 48, 6144, 4096, 16, none=0.1),
        # a mixed prefill batch of eight requests with rank-64 adapters, lengths uneven
        _lora("lora_glm_m4096", "lora", 4096, 8, 6144, 4096, 64, skew=1.0),
        # a fine-tuning step of four adapters at once, ragged row count
        _lora("lora_bwd_glm_m4001", "lora_backward", 4001, 4, 6144, 4096, 16, none=0.02, skew=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["permute", "permute_backward", "unpermute", "unpermute_backward",
                     "route_backward", "lora", "lora_backward"])
    if op.startswith("lora"):
        back = op == "lora_backward"
        G = _log(rng, 1, 8 if back else 64)
        r = 8 * _log(rng, 1, 8)
        K, N = 8 * _log(rng, 32, 768), 8 * _log(rng, 32, 512)
        M = _log(rng, 1, 4000)
        return dict(op=op, M=M, G=G, K=K, N=N, r=r, none=rng.choice([0.0, 0.0, 0.1, 0.5]),
                    skew=rng.choice([0.0, 0.5, 1.0]))
    E = _log(rng, 2, 256)
    k = rng.randint(1, min(8, E))
    H = rng.choice([_log(rng, 64, 6144), 64 * _log(rng, 1, 96)])
    M = _log(rng, 1, 8000 if op == "route_backward" else 4000)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if dtype == "fp32":
        H = min(H, 2560)
    if op == "unpermute_backward":      # reads and writes every row
        H = min(H, 1600 if dtype == "fp32" else 3200)
    local = rng.choice([0, 0, max(1, E // 4)]) if op != "route_backward" else 0
    return dict(op=op, M=M, k=k, E=E, H=H, dtype=dtype, local=local, skew=rng.choice([0.0, 1.0]))


def _lora_ids(case, gen):
    """Adapter of each row; -1: none. Requests' shares are uneven by exp(skew * N(0, 1))."""
    M, G = case["M"], case["G"]
    p = torch.exp(case["skew"] * torch.randn(G, device="cuda", generator=gen))
    ids = torch.multinomial(p, M, replacement=True, generator=gen).to(torch.int32)
    drop = torch.rand(M, device="cuda", generator=gen) < case["none"]
    return torch.where(drop, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std).to(dtype)

    op, M = case["op"], case["M"]
    s = {"case": case, "op": op}
    bf = torch.bfloat16
    if op.startswith("lora"):
        G, K, N, r = case["G"], case["K"], case["N"], case["r"]
        s["ids"] = _lora_ids(case, gen)
        s["x"] = normal(M, K, dtype=bf)
        # both matrices as a trained adapter has them: entries of 1/sqrt(fan-in)
        s["A"] = normal(G, r, K, dtype=bf, std=K ** -0.5)
        s["B"] = normal(G, N, r, dtype=bf, std=r ** -0.5)
        s["scale"] = 2.0 * torch.rand(G, device="cuda", generator=gen) + 0.25
        if op == "lora":
            s["base"] = normal(M, N, dtype=bf)
            s["y"] = torch.empty_like(s["base"])
            s["z"] = torch.zeros(M, r, device="cuda")
        else:
            s["dy"] = normal(M, N, dtype=bf)
            s["dbase"] = normal(M, K, dtype=bf)
            # z = x A^T as the forward left it
            g = torch.arange(G, device="cuda").repeat_interleave(r)
            z = s["x"].float() @ s["A"].float().view(G * r, K).t()
            z = torch.where(s["ids"][:, None] == g[None, :], z, 0.0)
            s["z"] = z.view(M, G, r).sum(1)
            s["dx"] = torch.empty_like(s["dbase"])
            s["dA"] = torch.empty(G, r, K, device="cuda")
            s["dB"] = torch.empty(G, N, r, device="cuda")
        return s
    k, E, H, dt = case["k"], case["E"], case["H"], DTYPES[case["dtype"]]
    logits = normal(M, E) + case["skew"] * normal(E)
    top = torch.topk(logits, k, dim=1)
    ids = top.indices.to(torch.int32)
    s["w"] = torch.softmax(top.values, dim=1)
    s["E"] = case["local"] or E
    if op == "route_backward":
        s["ids"], s["dw"] = ids, normal(M, k)
        s["dlogits"] = torch.empty(M, E, device="cuda")
        return s
    if op == "permute":
        s["ids"] = ids
        s["x"] = normal(M, H, dtype=dt)
        s["rows"] = torch.zeros(M * k, H, dtype=dt, device="cuda")
        s["sorted"] = torch.empty(M * k, dtype=torch.int32, device="cuda")
        s["slot_row"] = torch.empty(M, k, dtype=torch.int32, device="cuda")
        s["off"] = torch.empty(s["E"] + 1, dtype=torch.int32, device="cuda")
        return s
    # the row of every slot, as the permutation of the same ids left it
    flat = ids.reshape(-1).long()
    ok = flat < s["E"]
    order = torch.argsort(torch.where(ok, flat, s["E"]), stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(M * k, device="cuda")
    s["slot_row"] = torch.where(ok, row, -1).to(torch.int32).view(M, k)
    if op == "permute_backward":
        s["drows"] = normal(M * k, H, dtype=dt)
        s["dx"] = torch.empty(M, H, dtype=dt, device="cuda")
    elif op == "unpermute":
        s["rows"] = normal(M * k, H, dtype=dt)
        s["y"] = torch.empty(M, H, dtype=dt, device="cuda")
    else:
        s["rows"] = normal(M * k, H, dtype=dt)
        s["dy"] = normal(M, H, dtype=dt)
        s["drows"] = torch.zeros(M * k, H, dtype=dt, device="cuda")
        s["dw"] = torch.empty(M, k, device="cuda")
    return s


# ----------------------------------------------------------------------------
# the library's entry points
# ----------------------------------------------------------------------------

def _scratch(s, nbytes):
    """The workspace a program keeps beside its buffers, allocated at the first pass."""
    if "scratch" not in s:
        s["scratch"] = torch.empty(max(nbytes(), 256), dtype=torch.uint8, device="cuda")
    return s["scratch"]


def _run_own(s):
    import weight_only_quantized_moe_amd as hm
    c, op = s["case"], s["op"]
    if op == "permute":
        ws = _scratch(s, lambda: hm.moe_permute_scratch_bytes(c["M"], c["k"], s["E"]))
        hm.moe_permute(s["x"], s["ids"], s["E"], s["rows"], s["sorted"], s["slot_row"], s["off"], ws)
        return {"rows": s["rows"], "sorted": s["sorted"], "slot_row": s["slot_row"], "off": s["off"]}
    if op == "permute_backward":
        hm.moe_permute_backward(s["drows"], s["slot_row"], s["dx"])
        return {"dx": s["dx"]}
    if op == "unpermute":
        hm.moe_unpermute(s["rows"], s["slot_row"], s["w"], s["y"])
        return {"y": s["y"]}
    if op == "unpermute_backward":
        hm.moe_unpermute_backward(s["dy"], s["rows"], s["slot_row"], s["w"], s["drows"], s["dw"])
        return {"drows": s["drows"], "dw": s["dw"]}
    if op == "route_backward":
        hm.moe_route_backward(s["ids"], s["w"], s["dw"], s["dlogits"])
        return {"dlogits": s["dlogits"]}
    if op == "lora":
        ws = _scratch(s, lambda: hm.moe_lora_scratch_bytes(c["M"], c["G"], c["K"], c["N"], c["r"])[0])
        hm.moe_lora(s["x"], s["ids"], s["A"], s["B"], s["scale"], s["base"], s["y"], s["z"], ws)
        return {"y": s["y"], "z": s["z"]}
    ws = _scratch(s, lambda: hm.moe_lora_scratch_bytes(c["M"], c["G"], c["K"], c["N"], c["r"])[1])
    hm.moe_lora_backward(s["dy"], s["x"], s["z"], s["ids"], s["A"], s["B"], s["scale"], s["dbase"],
                         s["dx"], s["dA"], s["dB"], ws)
    return {"dx": s["dx"], "dA": s["dA"], "dB": s["dB"]}


# ----------------------------------------------------------------------------
# the plain form
# ----------------------------------------------------------------------------

def _plain_permute(s):
    ids, x, E = s["ids"], s["x"], s["E"]
    n, k = ids.numel(), ids.shape[1]
    flat = ids.reshape(-1).long()
    dropped = bool(s["case"]["local"])
    if dropped:
        ok = flat < E
        flat = torch.where(ok, flat, E)
    order = torch.argsort(flat, stable=True)
    place = torch.arange(n, device=x.device)
    row = torch.empty_like(order)
    row[order] = place
    counts = (flat[:, None] == torch.arange(E, device=x.device)[None, :]).sum(0)
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rows = x[order // k]
    if dropped:
        row = torch.where(ok, row, -1)
        held = place < off[-1]
        order = torch.where(held, order, -1)
        rows = torch.where(held[:, None], rows, 0.0)
    i32 = torch.int32
    return {"rows": rows, "sorted": order.to(i32), "slot_row": row.to(i32).view(-1, k), "off": off.to(i32)}


def _plain_gather(rows, slot_row):
    """fp32 [M, k, H]: every slot's row, zero for a dropped slot."""
    M, k = slot_row.shape
    r = slot_row.reshape(-1).long()
    g = rows[r.clamp(min=0)].float().view(M, k, -1)
    return torch.where((slot_row >= 0)[..., None], g, 0.0)


def _plain_lora(s):
    ids, x, A, B, scale = s["ids"].long(), s["x"].float(), s["A"], s["B"], s["scale"]
    G, r, K = A.shape
    held = ids >= 0
    if x.shape[0] <= GATHER_ROWS:
        own_ids = ids.clamp(min=0)
        z = torch.where(held[:, None], (A[own_ids].float() * x[:, None, :]).sum(-1), 0.0)
        d = (B[own_ids].float() * (scale[own_ids][:, None] * z)[:, None, :]).sum(-1)
        return {"y": (s["base"].float() + d).to(s["base"].dtype), "z": z}
    g = torch.arange(G, device=x.device).repeat_interleave(r)
    z = torch.where(ids[:, None] == g[None, :], x @ A.float().view(G * r, K).t(), 0.0)
    d = (z * scale[g]) @ B.float().transpose(1, 2).reshape(G * r, -1)
    return {"y": (s["base"].float() + d).to(s["base"].dtype), "z": z.view(-1, G, r).sum(1)}


def _plain_lora_backward(s):
    ids, x, dy, A, B = s["ids"].long(), s["x"].float(), s["dy"].float(), s["A"], s["B"]
    G, r, K = A.shape
    g = torch.arange(G, device=x.device).repeat_interleave(r)
    mine = ids[:, None] == g[None, :]
    Bt = B.float().transpose(1, 2).reshape(G * r, -1)
    dz = torch.where(mine, (dy @ Bt.t()) * s["scale"][g], 0.0)
    sz = torch.where(mine, s["z"].repeat(1, G) * s["scale"][g], 0.0)
    dx = s["dbase"].float() + dz @ A.float().view(G * r, K)
    dA = (dz.t() @ x).view(G, r, K)
    dB = (sz.t() @ dy).view(G, r, -1).transpose(1, 2).contiguous()
    return {"dx": dx.to(s["dbase"].dtype), "dA": dA, "dB": dB}


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "permute":
        return _plain_permute(s)
    if op == "permute_backward":
        return {"dx": _plain_gather(s["drows"], s["slot_row"]).sum(1).to(s["drows"].dtype)}
    if op == "unpermute":
        y = (_plain_gather(s["rows"], s["slot_row"]) * s["w"][..., None]).sum(1)
        return {"y": y.to(s["rows"].dtype)}
    if op == "unpermute_backward":
        sr, dy = s["slot_row"], s["dy"].float()
        dw = (_plain_gather(s["rows"], sr) * dy[:, None, :]).sum(-1)
        d = (s["w"][..., None] * dy[:, None, :]).to(s["rows"].dtype).view(sr.numel(), -1)
        # one row more takes what the dropped slots would write
        drows = torch.zeros(sr.numel() + 1, d.shape[1], dtype=d.dtype, device=d.device)
        drows[torch.where(sr >= 0, sr, sr.numel()).reshape(-1).long()] = d
        return {"drows": drows[:-1], "dw": dw}
    if op == "route_backward":
        w, dw = s["w"], s["dw"]
        d = w * (dw - (w * dw).sum(-1, keepdim=True))
        dl = torch.zeros(w.shape[0], s["case"]["E"], device=w.device)
        return {"dlogits": dl.scatter_add(1, s["ids"].long(), d)}
    if op == "lora":
        return _plain_lora(s)
    return _plain_lora_backward(s)


# ----------------------------------------------------------------------------
# what a pass cannot do without, and the values in 64 bits
# ----------------------------------------------------------------------------

def work(case):
    op, M = case["op"], case["M"]
    if op.startswith("lora"):
        G, K, N, r = case["G"], case["K"], case["N"], case["r"]
        live = M * (1.0 - case["none"])             # rows with an adapter
        used = G * (1.0 - (1.0 - 1.0 / G) ** live)  # adapters that some row uses, even use
        mats = used * r * (K + N) * 2
        if op == "lora":
            return {"bytes": live * K * 2 + 2 * M * N * 2 + mats + M * r * 4 + M * 4,
                    "flops": 2 * live * r * (K + N)}
        return {"bytes": live * (K + N) * 2 + 2 * M * K * 2 + live * r * 4 + mats
                + G * r * (K + N) * 4 + M * 4,
                "flops": 4 * live * r * (K + N)}
    k, E, H, e = case["k"], case["E"], case["H"], SIZE[case["dtype"]]
    if op == "route_backward":
        return {"bytes": M * k * 12 + M * E * 4, "flops": 4 * M * k}
    share = (case["local"] or E) / E                # slots whose expert is held here
    n = M * k
    rows = n * share * H * e
    if op == "permute":
        return {"bytes": M * H * e + rows + 3 * n * 4, "flops": 0}
    if op == "unpermute_backward":
        return {"bytes": 2 * rows + M * H * e + 3 * n * 4, "flops": 3 * n * share * H}
    return {"bytes": rows + M * H * e + n * (8 if op == "unpermute" else 4),
            "flops": 2 * n * share * H}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    f64 = torch.float64
    if op == "permute":
        ids = s["ids"].reshape(-1).cpu().tolist()
        E, k = s["E"], case["k"]
        of = [[] for _ in range(E)]
        for slot, e in enumerate(ids):
            if 0 <= e < E:
                of[e].append(slot)
        order = [slot for run_of in of for slot in run_of]
        off = [0]
        for run_of in of:
            off.append(off[-1] + len(run_of))
        row = [-1] * len(ids)
        for at, slot in enumerate(order):
            row[slot] = at
        token = torch.tensor([slot // k for slot in order], dtype=torch.long, device="cuda")
        rows = torch.zeros(len(ids), case["H"], dtype=f64, device="cuda")
        rows[: len(order)] = s["x"].to(f64).index_select(0, token)
        i32 = dict(dtype=torch.int32, device="cuda")
        return {"rows": rows, "sorted": torch.tensor(order + [-1] * (len(ids) - len(order)), **i32),
                "slot_row": torch.tensor(row, **i32).view(-1, k), "off": torch.tensor(off, **i32)}
    if op == "route_backward":
        w, dw = s["w"].to(f64), s["dw"].to(f64)
        # (diag(w) - w w^T) dw, token by token
        d = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        d = (d * dw[:, None, :]).sum(-1)
        out = torch.zeros(case["M"], case["E"], dtype=f64, device="cuda")
        for j in range(case["k"]):
            out[torch.arange(case["M"], device="cuda"), s["ids"][:, j].long()] += d[:, j]
        return {"dlogits": out}
    if op in ("permute_backward", "unpermute"):
        src = (s["drows"] if op == "permute_backward" else s["rows"])
        acc = torch.zeros(case["M"], case["H"], dtype=f64, device="cuda")
        for j in range(case["k"]):
            r = s["slot_row"][:, j].long()
            t = torch.nonzero(r >= 0).reshape(-1)
            part = src[r[t]].to(f64)
            acc[t] += part if op == "permute_backward" else part * s["w"][t, j].to(f64)[:, None]
        return {"dx" if op == "permute_backward" else "y": acc}
    if op == "unpermute_backward":
        dy = s["dy"].to(f64)
        dr = torch.zeros(s["rows"].shape, dtype=f64, device="cuda")
        dw = torch.zeros(case["M"], case["k"], dtype=f64, device="cuda")
        for j in range(case["k"]):
            r = s["slot_row"][:, j].long()
            t = torch.nonzero(r >= 0).reshape(-1)
            dr[r[t]] = dy[t] * s["w"][t, j].to(f64)[:, None]
            dw[t, j] = (s["rows"][r[t]].to(f64) * dy[t]).sum(-1)
        return {"drows": dr, "dw": dw}
    G = case["G"]
    x, A, B, sc = s["x"].to(f64), s["A"].to(f64), s["B"].to(f64), s["scale"].to(f64)
    if op == "lora":
        y, z = s["base"].to(f64), torch.zeros(case["M"], case["r"], dtype=f64, device="cuda")
        for g in range(G):
            t = torch.nonzero(s["ids"] == g).reshape(-1)
            z[t] = torch.mm(x[t], A[g].t().contiguous())
            y[t] += sc[g] * torch.mm(z[t], B[g].t().contiguous())
        return {"y": y, "z": z}
    dy, z = s["dy"].to(f64), s["z"].to(f64)
    dx, dA, dB = s["dbase"].to(f64), torch.zeros_like(A), torch.zeros_like(B)
    for g in range(G):
        t = torch.nonzero(s["ids"] == g).reshape(-1)
        dz = sc[g] * torch.mm(dy[t], B[g])
        dx[t] += torch.mm(dz, A[g])
        dA[g] = torch.mm(dz.t().contiguous(), x[t])
        dB[g] = sc[g] * torch.mm(dy[t].t().contiguous(), z[t])
    return {"dx": dx, "dA": dA, "dB": dB}
