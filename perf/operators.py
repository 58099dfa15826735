"""Cases of the token-sorting and low-rank-adapter operators beside the MoE layer, with
their plain forms.

``run`` makes one pass through one operator: in its plain form (elementary torch
operations in 32 bits) or, with ``own`` set, through the library.  ``exact`` computes the
same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token sent to its 8 experts (the decode layer's shape): launch latency
        dict(name="sort_t1", op="sort", T=1, H=6144, E=256, k=8, type="f16", align=1, topp=False),
        # a long prompt's tokens laid out for a grouped product whose tiles hold 16 rows
        dict(name="sort_t2048", op="sort", T=2048, H=6144, E=256, k=8, type="bf16", align=16, topp=False),
        # gradient of a small batch's sorted rows, some experts dropped by top-p
        dict(name="sort_bwd_t16", op="sort_bwd", T=16, H=2048, E=256, k=8, type="f16", to="f16", align=1, topp=True),
        # gradient of a training batch's sorted rows
        dict(name="sort_bwd_t2048", op="sort_bwd", T=2048, H=6144, E=256, k=8, type="bf16", to="bf16", align=16,
             topp=False),
        # eight decoded tokens: fp32 expert rows weighted and summed onto the shared expert's
        dict(name="unsort_t8", op="unsort", T=8, H=6144, E=256, k=8, type="f32", to="f16", align=1, topp=False,
             shared=True),
        # a long prompt's expert rows weighted and summed
        dict(name="unsort_t2048", op="unsort", T=2048, H=6144, E=256, k=8, type="bf16", to="bf16", align=16,
             topp=False, shared=False),
        # a ragged small batch: gradients of rows and combine weights
        dict(name="unsort_bwd_t37", op="unsort_bwd", T=37, H=6144, E=256, k=8, type="f16", align=1, topp=True),
        # a training batch: gradients of rows and combine weights
        dict(name="unsort_bwd_t2048", op="unsort_bwd", T=2048, H=6144, E=256, k=8, type="bf16", align=16, topp=False),
        # eight users decoding, each with an adapter out of 64, beside the fp32 shared projection
        dict(name="adapters_t8", op="adapters", T=8, K=6144, N=6144, n=64, r=16, type="f16", to="f32", seqs=8,
             save=False),
        # prompts of 24 requests with 8 adapters of rank up to 64
        dict(name="adapters_t4096", op="adapters", T=4096, K=6144, N=6144, n=8, r=64, type="bf16", to="bf16", seqs=24,
             save=True),
        # a small fine-tuning batch of two sequences, narrow layer
        dict(name="adapters_bwd_t200", op="adapters_bwd", T=200, K=2048, N=512, n=2, r=8, type="f16", to="f16",
             seqs=2),
        # a fine-tuning batch over four adapters
        dict(name="adapters_bwd_t4096", op="adapters_bwd", T=4096, K=6144, N=6144, n=4, r=32, type="bf16", to="bf16",
             seqs=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "sort_bwd", "unsort", "unsort_bwd", "adapters", "adapters_bwd"])
    if op.startswith("adapters"):
        n = _log(rng, 1, 64)
        r = 8 * rng.randint(1, min(8, 1024 // (8 * n)))
        T = _log(rng, 1, 4096)
        c = dict(op=op, T=T, K=8 * _log(rng, 8, 768), N=8 * _log(rng, 4, 768), n=n, r=r,
                 type=rng.choice(["f16", "bf16"]), seqs=min(T, _log(rng, 1, 256)))
        if op == "adapters":
            c["to"] = rng.choice([c["type"], "f32"])
            c["save"] = rng.random() < 0.5
            if c["to"] == "f32" and rng.random() < 0.5:
                c["N"] = rng.randint(5, 256)      # logits of any number of experts
        else:
            c["to"] = rng.choice([c["type"], "f32"])
        return c
    E = _log(rng, 4, 256)
    c = dict(op=op, T=_log(rng, 1, 2048), H=64 * _log(rng, 4, 96), E=E, k=rng.randint(1, min(8, E)),
             type=rng.choice(["f16", "bf16", "f32"]), align=rng.choice([1, 1, 8, 16, 24, 64]),
             topp=rng.random() < 0.3)
    if c["type"] == "f32":
        c["T"] = min(c["T"], 1000)
    c["align"] = 1 if E * c["align"] > 4 * c["T"] * c["k"] else c["align"]
    if op in ("sort_bwd", "unsort"):
        c["to"] = rng.choice(sorted({c["type"], "f16", "bf16"}))
    if op == "unsort":
        c["shared"] = rng.random() < 0.5
    return c


def _rows(c):
    """Rows a sorted buffer must have: every segment may end in align - 1 rows of padding."""
    a = c["T"] * c["k"]
    return a + min(c["E"], a) * (c["align"] - 1)


# ------------------------------------------------------------------------------ inputs
def _routing(c, g):
    """Distinct experts per token under a skewed preference; top-p leaves -1 at the end."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn((T, E), generator=g, device=DEV) + 1.5 * torch.rand((E,), generator=g, device=DEV)
    score, idx = torch.topk(torch.sigmoid(logits), k, dim=1)
    keep = torch.full((T, 1), k, device=DEV)
    if c["topp"]:
        keep = torch.randint(1, k + 1, (T, 1), generator=g, device=DEV)
    on = torch.arange(k, device=DEV)[None, :] < keep
    score = torch.where(on, score, torch.zeros_like(score))
    w = 2.5 * score / score.sum(1, keepdim=True)
    return torch.where(on, idx, torch.full_like(idx, -1)).to(torch.int32), w


def _positions(idx, E, align):
    """row_of [T, k], counts [E], seg_offsets [E + 1] of a stable sort by expert."""
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.argsort(key, stable=True)
    sorted_key = key[order]
    start = torch.searchsorted(sorted_key, torch.arange(E + 1, device=DEV))
    counts = start[1:] - start[:-1]
    seg = torch.zeros(E + 1, dtype=torch.long, device=DEV)
    seg[1:] = torch.cumsum((counts + align - 1) // align * align, 0)
    row_of = torch.empty_like(flat)
    row_of[order] = torch.arange(flat.numel(), device=DEV) - start[sorted_key] + seg[sorted_key]
    row_of = torch.where(flat < 0, torch.full_like(flat, -1), row_of)
    return row_of.reshape(idx.shape).to(torch.int32), counts.to(torch.int32), seg.to(torch.int32)


def _requests(c, g):
    """adapter_of [T]: contiguous requests of ragged lengths, one in ten without an adapter."""
    T, n, seqs = c["T"], c["n"], c["seqs"]
    cut = torch.rand(seqs, generator=g, device=DEV) + 0.05
    ends = torch.cumsum(cut, 0) / cut.sum() * T
    which = torch.randint(0, n, (seqs,), generator=g, device=DEV)
    which = torch.where(torch.rand(seqs, generator=g, device=DEV) < 0.1, torch.full_like(which, -1), which)
    seq = torch.searchsorted(ends, torch.arange(T, device=DEV).to(ends.dtype), right=True).clamp(max=seqs - 1)
    return which[seq].to(torch.int32)


def _layer(c):
    """The layer the rows belong to; its expert weights take no part here, so they are narrow."""
    import w4a16_quantized_expert_b200 as moe
    from w4a16_quantized_expert_b200.device import DeviceLayer
    H, E, I = c["H"], c["E"], 64
    z = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
    f = torch.float32
    t = {"Wr": z(E, H, t=f), "bias": z(E, t=f), "g": z(E, I, H // 2), "u": z(E, I, H // 2), "d": z(E, H, I // 2),
         "sg": z(E, I, t=f), "su": z(E, I, t=f), "sd": z(E, H, t=f)}
    d = {"H": H, "I": I, "I_sh": 0, "E": E, "k": c["k"], "n_shared": 0, "scaling": 2.5,
         "fmt": moe.MOE_FMT_INT4_ROWSCALE, "top_p": 0.5 if c["topp"] else 0.0}
    return DeviceLayer(d, max_tokens=c["T"], device=DEV, tensors=t)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rnd = lambda *s, t="f32": torch.randn(s, generator=g, device=DEV).to(TYPES[t])  # noqa: E731
    s = {"case": c}
    if c["op"].startswith("adapters"):
        T, K, N, n, r, ty = c["T"], c["K"], c["N"], c["n"], c["r"], c["type"]
        s["adapter_of"] = _requests(c, g)
        s["rank"] = torch.randint((r + 1) // 2, r + 1, (n,), generator=g, device=DEV).to(torch.int32)
        s["scaling"] = 0.5 + torch.rand(n, generator=g, device=DEV)
        s["a"] = (torch.randn((n, r, K), generator=g, device=DEV) / math.sqrt(K)).to(TYPES[ty])
        s["b"] = (torch.randn((n, N, r), generator=g, device=DEV) / math.sqrt(r)).to(TYPES[ty])
        s["x"] = rnd(T, K, t=ty)
        if c["op"] == "adapters":
            s["base"] = rnd(T, N, t=c["to"])       # the shared projection's output
            s["out"] = torch.empty_like(s["base"])
            s["z"] = torch.zeros((T, r), dtype=torch.float32, device=DEV) if c["save"] else None
        else:
            s["z"] = _shrink(s, s["x"], s["a"])    # what the forward pass kept
            s["dy"] = rnd(T, N, t=ty)
            s["base"] = rnd(T, K, t=c["to"])       # the shared projection's input gradient
            s["out"] = torch.empty_like(s["base"])
            s["da"] = torch.empty((n, r, K), dtype=torch.float32, device=DEV)
            s["db"] = torch.empty((n, N, r), dtype=torch.float32, device=DEV)
        if own:
            from w4a16_quantized_expert_b200.device import DeviceAdapters
            s["handle"] = DeviceAdapters(s["a"], s["b"], s["scaling"], s["rank"], max_tokens=T)
            s["ws"] = s["handle"].workspace(T)
        return s
    T, H, E, k, ty = c["T"], c["H"], c["E"], c["k"], c["type"]
    s["idx"], s["w"] = _routing(c, g)
    n = _rows(c)
    if c["op"] == "sort":
        s["x"] = rnd(T, H, t=ty)
        i32 = dict(dtype=torch.int32, device=DEV)
        s["out"] = (torch.zeros((n, H), dtype=TYPES[ty], device=DEV), torch.empty((T, k), **i32),
                    torch.empty(E, **i32), torch.empty(E + 1, **i32))
    else:
        s["row_of"], s["counts"], s["seg"] = _positions(s["idx"], E, c["align"])
        s["rows"] = rnd(n, H, t=ty)
        if c["op"] == "unsort_bwd":
            s["dy"] = rnd(T, H, t=ty)
            s["out"] = (torch.zeros((n, H), dtype=TYPES[ty], device=DEV),
                        torch.empty((T, k), dtype=torch.float32, device=DEV))
        else:
            s["shared"] = rnd(T, H) if c.get("shared") else None
            s["out"] = torch.empty((T, H), dtype=TYPES[c["to"]], device=DEV)
    if own:
        s["handle"] = _layer(c)
        s["ws"] = s["handle"].sort_workspace(T)
    return s


# ------------------------------------------------------------------------------ plain forms
def _own_block(s, r):
    """[T, n * r] mask of the columns of each token's adapter (all adapters' ranks laid side by side)."""
    n = s["rank"].numel()
    col = torch.arange(n * r, device=DEV)
    live = (col % r) < s["rank"].long()[col // r]
    return (s["adapter_of"].long()[:, None] == (col // r)[None, :]) & live[None, :]


def _shrink(s, x, a):
    """z [T, r] = A_a x of each token's own adapter."""
    n, r, K = a.shape
    z = x.float() @ a.float().reshape(n * r, K).t()
    z = torch.where(_own_block(s, r), z, torch.zeros_like(z))
    return z.reshape(-1, n, r).sum(1)


def _spread(s, z):
    """z [T, r] placed in its adapter's columns: [T, n * r]."""
    n, r = s["rank"].numel(), z.shape[1]
    wide = z.repeat(1, n)
    return torch.where(_own_block(s, r), wide, torch.zeros_like(wide))


def _scale(s):
    a = s["adapter_of"].long()
    return torch.where(a < 0, torch.zeros_like(s["scaling"][a]), s["scaling"][a])[:, None]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "adapters":
        n, N, r = s["b"].shape
        z = _shrink(s, s["x"], s["a"])
        delta = _spread(s, z * _scale(s)) @ s["b"].float().permute(0, 2, 1).reshape(n * r, N)
        y = (s["base"].float() + delta).to(s["base"].dtype)
        return (y, z) if c["save"] else y
    if op == "adapters_bwd":
        n, N, r = s["b"].shape
        K = c["K"]
        dy, x = s["dy"].float(), s["x"].float()
        dz = dy @ s["b"].float().permute(0, 2, 1).reshape(n * r, N).t()
        dz = torch.where(_own_block(s, r), dz, torch.zeros_like(dz)) * _scale(s)
        dx = (s["base"].float() + dz @ s["a"].float().reshape(n * r, K)).to(s["base"].dtype)
        da = (dz.t() @ x).reshape(n, r, K)
        db = (_spread(s, s["z"] * _scale(s)).t() @ dy).reshape(n, r, N).permute(0, 2, 1).contiguous()
        return dx, da, db
    if op == "sort":
        row_of, counts, seg = _positions(s["idx"], c["E"], c["align"])
        T, k = row_of.shape
        rows = torch.zeros((_rows(c) + 1, c["H"]), dtype=s["x"].dtype, device=DEV)   # the last row takes what is dropped
        to = torch.where(row_of < 0, torch.full_like(row_of, _rows(c)), row_of).long().reshape(-1)
        rows[to] = s["x"][torch.arange(T * k, device=DEV) // k]
        return rows[:-1], row_of, counts, seg
    row_of, w = s["row_of"], s["w"]
    live = row_of >= 0
    at = row_of.clamp(min=0).long()
    if op == "unsort_bwd":
        dy = s["dy"].float()
        dw = torch.where(live, (s["rows"][at].float() * dy[:, None, :]).sum(2), torch.zeros_like(w))
        rows = torch.zeros((s["rows"].shape[0] + 1, c["H"]), dtype=s["rows"].dtype, device=DEV)
        to = torch.where(live, row_of, torch.full_like(row_of, rows.shape[0] - 1)).long().reshape(-1)
        rows[to] = (w[:, :, None] * dy[:, None, :]).to(rows.dtype).reshape(-1, c["H"])
        return rows[:-1], dw
    by = torch.where(live, w if op == "unsort" else torch.ones_like(w), torch.zeros_like(w))
    y = (by[:, :, None] * s["rows"][at].float()).sum(1)
    if s["shared"] is not None:
        y = y + s["shared"]
    return y.to(s["out"].dtype)


def run(state):
    if not own:
        return _plain(state)
    s, c = state, state["case"]
    h, op = s["handle"], c["op"]
    if op == "adapters":
        y = h.apply(s["x"], s["adapter_of"], s["ws"], y_in=s["base"], y=s["out"], z=s["z"])
        return (y, s["z"]) if c["save"] else y
    if op == "adapters_bwd":
        return h.backward(s["x"], s["z"], s["dy"], s["adapter_of"], s["ws"], dx_in=s["base"], dx=s["out"],
                          da=s["da"], db=s["db"])
    if op == "sort":
        return h.sort_tokens(s["x"], s["idx"], s["ws"], align=c["align"], out=s["out"])
    if op == "sort_bwd":
        return h.sort_tokens_backward(s["rows"], s["row_of"], dx=s["out"])
    if op == "unsort":
        return h.unsort_tokens(s["rows"], s["row_of"], s["w"], y_shared=s["shared"], y=s["out"])
    return h.unsort_tokens_backward(s["dy"], s["rows"], s["row_of"], s["w"], s["counts"], s["seg"], out=s["out"])


# ------------------------------------------------------------------------------ floors
def work(case):
    c = case
    if c["op"].startswith("adapters"):
        T, K, N, r = c["T"], c["K"], c["N"], c["r"]
        used = min(c["n"], c["seqs"])
        b = T * K * 2 + T * 4 + used * r * (K + N) * 2
        if c["op"] == "adapters":
            return {"bytes": b + 2 * T * N * SIZE[c["to"]] + (T * r * 4 if c["save"] else 0),
                    "flops": 2 * T * r * (K + N)}
        return {"bytes": b + T * N * 2 + 2 * T * K * SIZE[c["to"]] + T * r * 4 + c["n"] * r * (K + N) * 4,
                "flops": 4 * T * r * (K + N)}
    T, H, k, z = c["T"], c["H"], c["k"], SIZE[c["type"]]
    kept = T * (k + 1) / 2 if c["topp"] else T * k      # top-p keeps a uniform 1 .. k of each token's experts
    if c["op"] == "sort":
        return {"bytes": T * H * z + kept * H * z + T * k * 8 + c["E"] * 8, "flops": 0}
    if c["op"] == "unsort_bwd":
        return {"bytes": T * H * z + 2 * kept * H * z + T * k * 12, "flops": 3 * kept * H}
    b = kept * H * z + T * H * SIZE[c["to"]] + T * k * 4
    if c["op"] == "unsort":
        b += T * k * 4 + (T * H * 4 if c["shared"] else 0)
    return {"bytes": b, "flops": 2 * kept * H}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], s["case"]["op"]
    f = torch.float64
    if op.startswith("adapters"):
        n, r = c["n"], c["r"]
        x = s["x"].to(f)
        out = s["base"].to(f).clone()
        z = torch.zeros((c["T"], r), dtype=f, device=DEV)
        da = torch.zeros((n, r, c["K"]), dtype=f, device=DEV)
        db = torch.zeros((n, c["N"], r), dtype=f, device=DEV)
        which, rank, scaling = s["adapter_of"].tolist(), s["rank"].tolist(), s["scaling"].tolist()
        for i in range(n):
            t = [j for j, v in enumerate(which) if v == i]
            if not t:
                continue
            q, t = rank[i], torch.tensor(t, device=DEV)
            A, B = s["a"][i, :q].to(f), s["b"][i, :, :q].to(f)
            if op == "adapters":
                z[t, :q] = x[t] @ A.t()
                out[t] += scaling[i] * (z[t, :q] @ B.t())
            else:
                dy = s["dy"][t].to(f)
                dz = scaling[i] * (dy @ B)
                out[t] += dz @ A
                da[i, :q] = dz.t() @ x[t]
                db[i, :, :q] = scaling[i] * (dy.t() @ s["z"][t, :q].to(f))
        if op == "adapters":
            return (out, z) if c["save"] else out
        return out, da, db
    T, k, H, E, align = c["T"], c["k"], c["H"], c["E"], c["align"]
    idx = s["idx"].tolist()
    members = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if idx[t][j] >= 0:
                members[idx[t][j]].append(t * k + j)
    seg, row_of = [0], [-1] * (T * k)
    for m in members:
        for i, a in enumerate(m):
            row_of[a] = seg[-1] + i
        seg.append(seg[-1] + -(-len(m) // align) * align)
    at = torch.tensor([r for r in row_of if r >= 0], device=DEV)
    a = torch.tensor([i for i, r in enumerate(row_of) if r >= 0], device=DEV)
    if op == "sort":
        rows = torch.zeros((_rows(c), H), dtype=f, device=DEV)
        rows[at] = s["x"].to(f)[a // k]
        i32 = dict(dtype=torch.int32, device=DEV)
        return (rows, torch.tensor(row_of, **i32).reshape(T, k), torch.tensor([len(m) for m in members], **i32),
                torch.tensor(seg, **i32))
    w = s["w"].to(f).reshape(-1)
    if op == "unsort_bwd":
        dy = s["dy"].to(f)[a // k]
        rows = torch.zeros((_rows(c), H), dtype=f, device=DEV)
        rows[at] = w[a, None] * dy
        dw = torch.zeros(T * k, dtype=f, device=DEV)
        dw[a] = (dy * s["rows"][at].to(f)).sum(1)
        return rows, dw.reshape(T, k)
    y = s["shared"].to(f).clone() if s["shared"] is not None else torch.zeros((T, H), dtype=f, device=DEV)
    v = s["rows"][at].to(f)
    return y.index_add_(0, a // k, v * w[a, None] if op == "unsort" else v)
