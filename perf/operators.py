"""Cases, plain forms and exact values of the operators on the paged key-value cache.

Three operators share one cache of pages:

  store   projected rows of tokens of many sequences -> bias, optional q/k norm of each head, neox
          rotation, q out, k and v into the cache's pages (qkv_paged_store_step)
  attn    one new token of every sequence attends over its cached slots, optionally adding each
          slot's attention weight to a running sum (qkv_attn_step)
  evict   every (sequence, kv head) keeps the slots with the largest running sums and the newest
          ones, and fills the freed slots from behind (qkv_evict_step)

Head layouts are those of qkv_rope_kv_gb300.configs (14/2/64, 28/4/128, 40/8/128); drawn cases
vary them.  Slot s of sequence b is row s % page of page table[b, s // page].
"""
import math
import random

import torch

own = False

THETA = 1.0e6
EPS = 1.0e-6
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # attention of a single short f32 sequence (the 0.5B layer's own cache): latency only
        dict(name="attn-0.5b-b1-short", op="attn", nh=14, nkv=2, hd=64, kv="f32", page=16, batch=1, length=509,
             ragged=False, window=0, weights=False, out="f32"),
        # one user's chat turn on the 7B layout: too few heads to fill the GPU without splitting the length
        dict(name="attn-7b-b1", op="attn", nh=28, nkv=4, hd=128, kv="f16", page=16, batch=1, length=1641,
             ragged=False, window=0, weights=False, out="f32"),
        # one long document on the 14B layout
        dict(name="attn-14b-b1-long", op="attn", nh=40, nkv=8, hd=128, kv="f16", page=64, batch=1, length=32749,
             ragged=False, window=0, weights=False, out="bf16"),
        # a serving batch of uneven sequences on the 14B layout
        dict(name="attn-14b-b64", op="attn", nh=40, nkv=8, hd=128, kv="f16", page=16, batch=64, length=8192,
             ragged=True, window=0, weights=False, out="bf16"),
        # a serving batch that also keeps the running sums that eviction goes by
        dict(name="attn-7b-b32-weights", op="attn", nh=28, nkv=4, hd=128, kv="f16", page=32, batch=32, length=4099,
             ragged=True, window=0, weights=True, out="f32"),
        # one decode token of one 0.5B sequence, and of a 14B batch with q/k norms, and a long prompt
        dict(name="store-0.5b-t1", op="store", nh=14, nkv=2, hd=64, kv="f32", page=16, mode="decode", tokens=1,
             y="f32", norm=False),
        dict(name="store-14b-t64-norm", op="store", nh=40, nkv=8, hd=128, kv="f16", page=16, mode="decode", tokens=64,
             y="f32", norm=True),
        dict(name="store-14b-t8191-norm", op="store", nh=40, nkv=8, hd=128, kv="f16", page=64, mode="prompt",
             tokens=8191, y="bf16", norm=True),
        # eviction of the 64 slots that a running 14B batch gained since the last time
        dict(name="evict-14b-b8-step", op="evict", nh=40, nkv=8, hd=128, kv="f16", page=16, batch=8, length=2112,
             budget=2048, recent=256, ragged=False),
        # a long prompt cut down to its budget after prefill
        dict(name="evict-7b-b1-prompt", op="evict", nh=28, nkv=4, hd=128, kv="f16", page=64, batch=1, length=32749,
             budget=8192, recent=512, ragged=False),
        # an uneven batch, some of its sequences still below their budget, in f32
        dict(name="evict-0.5b-b32-ragged", op="evict", nh=14, nkv=2, hd=64, kv="f32", page=32, batch=32, length=4099,
             budget=1000, recent=100, ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "store", "evict"])
    nkv = rng.choice([1, 2, 4, 5, 8])
    c = dict(op=op, nh=nkv * rng.choice([1, 2, 4, 5, 7, 8, 12]), nkv=nkv, hd=rng.choice([64, 64, 80, 96, 128, 128, 256]),
             kv=rng.choice(["f16", "f16", "f32"]), page=rng.choice([1, 8, 16, 17, 32, 64, 128, 256]))
    if op == "store":
        c.update(mode=rng.choice(["decode", "prompt"]), y=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.6)
        most = 8191 * 7168 // ((c["nh"] + 2 * nkv) * c["hd"])
        c["tokens"] = _log(rng, 1, min(256 if c["mode"] == "decode" else 8191, most))
        return c
    # no more cached values than a quarter of the largest listed case
    room = (1 << 27) // (nkv * c["hd"])
    c["batch"] = _log(rng, 1, 128)
    c["ragged"] = rng.random() < 0.7
    if op == "attn":
        c["length"] = _log(rng, 1, max(1, min(40000, room // c["batch"])))
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        c["weights"] = rng.random() < 0.4
        c["out"] = rng.choice(["f32", "bf16"])
    else:
        c["length"] = _log(rng, 8, max(8, min(40000, room // c["batch"])))
        c["budget"] = _log(rng, 1, c["length"])
        c["recent"] = rng.randint(0, c["budget"])
    return c


# ---------------------------------------------------------------- inputs

def _cache(case, gen, r, batch, cap):
    """Pools, table: every sequence has pages for `cap` slots, scattered over the pool; all rows hold numbers."""
    ps, nkv, hd = case["page"], case["nkv"], case["hd"]
    per = -(-cap // ps)
    n_pages = batch * per + 3
    table = torch.randperm(n_pages, generator=gen, device="cuda")[:batch * per].to(torch.int32).view(batch, per)
    pools = [torch.empty(n_pages, ps, nkv * hd, dtype=DT[case["kv"]], device="cuda") for _ in range(2)]
    for p in pools:
        p.normal_(generator=gen)
    return dict(k=pools[0], v=pools[1], table=table.contiguous(), cap=per * ps)


def _lengths(case, r):
    B, L = case["batch"], case["length"]
    lens = [r.randint(0, L) if case["ragged"] else L for _ in range(B)]
    lens[r.randrange(B)] = L
    return lens


def _dev(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "store":
        nt, ps = case["tokens"], case["page"]
        if case["mode"] == "decode":  # token t is the newest of sequence t
            batch, cap = nt, max(ps, 64)
            pos = [r.randint(0, 30000) for _ in range(nt)]
            seqs, slots = list(range(nt)), [r.randrange(cap) for _ in range(nt)]
        else:  # one sequence's prompt behind what it has cached
            batch, first = 1, r.randint(0, 2000)
            cap = 2000 + nt
            pos = list(range(first, first + nt))
            seqs, slots = [0] * nt, pos
        st = _cache(case, gen, r, batch, cap)
        R = (nh + 2 * nkv) * hd
        st["y"] = rand(nt, R).to(DT[case["y"]])
        st["bias"] = 0.1 * rand(R)
        st["qw"], st["kw"] = (1 + 0.1 * rand(hd), 1 + 0.1 * rand(hd)) if case["norm"] else (None, None)
        st["pos"], st["seqs"], st["slots"] = _dev(pos), _dev(seqs), _dev(slots)
        st["q"] = torch.empty(nt, nh * hd, device="cuda")
        st["inv"] = _dev([THETA ** (-2.0 * d / hd) for d in range(hd // 2)], torch.float32)
        return st
    lens = _lengths(case, r)
    st = _cache(case, gen, r, case["batch"], case["length"])
    st["lens"], B, cap = _dev(lens), case["batch"], st["cap"]
    if case["op"] == "attn":
        st["q"] = 2.0 * rand(B, nh * hd)
        st["out"] = torch.empty(B, nh * hd, dtype=DT[case["out"]], device="cuda")
        st["weight"] = torch.rand(B, nkv, cap, generator=gen, device="cuda") if case["weights"] else None
        return st
    # weights as attention leaves them: most of the mass on few slots, some never attended to
    w = torch.exp(2.0 * rand(B, nkv, cap))
    st["weight"] = torch.where(w < 0.1, 0.0, w)
    # slot_pos: the slots below the budget were filled in any order, the others follow in order
    low = min(case["budget"], cap)
    order = torch.rand(B, nkv, low, generator=gen, device="cuda").argsort(-1)
    st["pos"] = torch.cat([order, torch.arange(low, cap, device="cuda").expand(B, nkv, cap - low)], -1).int().contiguous()
    st["next"] = st["lens"].clone()
    st["lens_out"] = torch.zeros_like(st["lens"])
    st["weight_out"], st["pos_out"] = st["weight"].clone(), st["pos"].clone()
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        import qkv_rope_kv_gb300 as Q
        kv = {"f32": Q.QKV_F32, "f16": Q.QKV_F16}[case["kv"]]
        plan = Q.qkv_plan_create(case["nh"] * case["hd"], case["nh"], case["nkv"], case["hd"], THETA, st["cap"],
                                 w_dtype=Q.QKV_BF16, kv_dtype=kv)
        track = {} if case["op"] == "store" else dict(slot_weight=st["weight"], slot_pos=st.get("pos"))
        cache = Q.PagedKv(plan, st["k"], st["v"], st["table"], **track)
        st.update(Q=Q, plan=plan, cache=cache)
        if case["op"] == "attn":
            st["ws"] = torch.zeros(Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
        if case["op"] == "evict":
            st["ws"] = torch.zeros(Q.qkv_evict_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return {"store": _store, "attn": _attn, "evict": _evict}[st["case"]["op"]](st)


def _rows(st, slots, batch_index):
    """Row numbers in the pools, seen as [pages * page, nkt], of `slots` of the sequences `batch_index`."""
    ps = st["case"]["page"]
    slots = slots.long()
    return st["table"].long()[batch_index, slots // ps] * ps + slots % ps


def _store(st):
    c = st["case"]
    if own:
        st["Q"].qkv_paged_store_step(st["plan"], st["cache"], st["y"], st["bias"], st["qw"], st["kw"], EPS, st["pos"],
                                     st["seqs"], st["slots"], st["q"])
        return {"q": st["q"], "k": st["k"], "v": st["v"]}
    nh, nkv, hd, nt = c["nh"], c["nkv"], c["hd"], c["tokens"]
    z = (st["y"].float() + st["bias"]).view(nt, nh + 2 * nkv, hd)
    qk, v = z[:, :nh + nkv], z[:, nh + nkv:]
    if c["norm"]:
        w = torch.cat([st["qw"].expand(nh, hd), st["kw"].expand(nkv, hd)])
        qk = qk / torch.sqrt(qk.square().mean(-1, keepdim=True) + EPS) * w
    # the stage's angle is one f32 value, the rounded product of position and table entry
    angle = (st["pos"].double()[:, None] * st["inv"].double()).float()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    x0, x1 = qk[..., :hd // 2], qk[..., hd // 2:]
    qk = torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1)
    st["q"].copy_(qk[:, :nh].reshape(nt, -1))
    rows = _rows(st, st["slots"], st["seqs"].long())
    st["k"].view(-1, nkv * hd)[rows] = qk[:, nh:].reshape(nt, -1).to(st["k"].dtype)
    st["v"].view(-1, nkv * hd)[rows] = v.reshape(nt, -1).to(st["v"].dtype)
    return {"q": st["q"], "k": st["k"], "v": st["v"]}


def _attn(st):
    c = st["case"]
    scale = c["hd"] ** -0.5
    if own:
        st["Q"].qkv_attn_step(st["plan"], st["cache"], st["q"], st["lens"], scale, st["out"], st["ws"],
                              window=c["window"], add_weight=c["weights"])
        return {"out": st["out"], "weight": st["weight"]} if c["weights"] else {"out": st["out"]}
    B, L, nh, nkv, hd = c["batch"], c["length"], c["nh"], c["nkv"], c["hd"]
    slots = torch.arange(L, device="cuda").expand(B, L)
    rows = _rows(st, slots, torch.arange(B, device="cuda")[:, None])
    K = st["k"].view(-1, nkv, hd)[rows].float().permute(0, 2, 3, 1)  # [B, nkv, hd, L]
    V = st["v"].view(-1, nkv, hd)[rows].float().transpose(1, 2)      # [B, nkv, L, hd]
    q = st["q"].view(B, nkv, nh // nkv, hd) * scale
    n = st["lens"][:, None]
    seen = slots < n
    if c["window"]:
        seen = seen & (slots >= n - c["window"])
    seen = seen[:, None, None]
    s = torch.where(seen, q @ K, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    st["out"].copy_((p @ V).reshape(B, nh * hd))
    if not c["weights"]:
        return {"out": st["out"]}
    st["weight"][..., :L] += p.sum(2)
    return {"out": st["out"], "weight": st["weight"]}


def _evict(st):
    c = st["case"]
    if own:
        st["Q"].qkv_evict_step(st["plan"], st["cache"], st["lens"], st["next"], c["budget"], c["recent"], st["lens_out"],
                               st["weight_out"], st["pos_out"], st["ws"])
        return {x: st[x] for x in ("k", "v", "lens_out", "weight_out", "pos_out")}
    B, nkv, hd, budget, cap = c["batch"], c["nkv"], c["hd"], c["budget"], st["cap"]
    n = st["lens"].long()[:, None, None]
    slot = torch.arange(cap, device="cuda")
    key = torch.where(st["pos"] >= (st["next"] - c["recent"])[:, None, None], math.inf, st["weight"])
    key = torch.where(slot < n, key, -1.0)
    best = key.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.zeros(B, nkv, cap, dtype=torch.bool, device="cuda").scatter_(-1, best, True) & (slot < n)
    over = n > budget
    holes, movers = over & ~kept & (slot < budget), over & kept & (slot >= budget)
    most = min(budget, cap - min(budget, cap))
    # i-th hole and i-th mover; places past the last pair copy a slot that no pair writes onto itself
    idle = torch.where(over, min(budget, cap - 1), 0)
    pairs = torch.arange(most, device="cuda") < holes.sum(-1, keepdim=True)
    to = torch.where(pairs, torch.where(holes, slot, cap + slot).sort(-1).values[..., :most], idle)
    at = torch.where(pairs, torch.where(movers, slot, cap + slot).sort(-1).values[..., :most], idle)
    b = torch.arange(B, device="cuda")[:, None, None]
    head = torch.arange(nkv, device="cuda")[:, None]
    row_to, row_at = _rows(st, to, b), _rows(st, at, b)
    for x in ("k", "v"):
        pool = st[x].view(-1, nkv, hd)
        pool[row_to, head] = pool[row_at, head]
    below = slot < torch.minimum(n, torch.full_like(n, budget))
    for x in ("weight", "pos"):
        moved = st[x].scatter(-1, to, st[x].gather(-1, at))
        st[x + "_out"].copy_(torch.where(below, moved, st[x + "_out"]))
    st["lens_out"].copy_(st["lens"].clamp(max=budget))
    return {x: st[x] for x in ("k", "v", "lens_out", "weight_out", "pos_out")}


# ---------------------------------------------------------------- what a pass cannot do without

def _mean_length(case):
    # listed and drawn batches: one full sequence, the others uniform between 0 and it
    B, L = case["batch"], case["length"]
    return (L + (B - 1) * L / 2) / B if case["ragged"] else L


def work(case):
    nh, nkv, hd, e = case["nh"], case["nkv"], case["hd"], SIZE[case["kv"]]
    if case["op"] == "store":
        nt, R = case["tokens"], (nh + 2 * nkv) * hd
        return {"bytes": nt * (R * SIZE[case["y"]] + 4 * nh * hd + 2 * nkv * hd * e + 16) + 4 * R,
                "flops": nt * R * 8}
    B, n = case["batch"], _mean_length(case)
    if case["op"] == "attn":
        n = min(n, case["window"]) if case["window"] else n
        each = 2 * n * nkv * hd * e + nh * hd * (4 + SIZE[case["out"]]) + 4 * n / case["page"] + 4
        return {"bytes": B * (each + (8 * n * nkv if case["weights"] else 0)), "flops": B * 4 * n * nh * hd}
    budget, recent = case["budget"], case["recent"]
    moved = 0.0
    if n > budget:
        older = n - recent
        moved = min(recent, n - budget) + (budget - recent) / max(older, 1) * max(0.0, older - budget)
    # weights and positions read, those kept written; each moved row of k and v read and written
    return {"bytes": B * nkv * (8 * n + 8 * min(n, budget) + moved * 4 * hd * e) + 12 * B, "flops": B * nkv * n}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = _inputs(case, seed)
    nh, nkv, hd, ps = case["nh"], case["nkv"], case["hd"], case["page"]
    table = st["table"].cpu().tolist()
    place = lambda b, s: table[b][s // ps] * ps + s % ps  # noqa: E731
    if case["op"] == "store":
        nt = case["tokens"]
        z = st["y"].double() + st["bias"].double()
        q, k, v = z.split([nh * hd, nkv * hd, nkv * hd], 1)
        angle = (st["pos"].float()[:, None] * st["inv"][None]).double()  # one f32 product, by definition
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]

        def finish(x, heads, w):
            x = x.reshape(nt, heads, hd)
            if case["norm"]:
                x = x * w.double() * (x.pow(2).sum(-1, keepdim=True) / hd + EPS).pow(-0.5)
            x = torch.complex(x[..., :hd // 2].contiguous(), x[..., hd // 2:].contiguous()) * turn
            return torch.cat([x.real, x.imag], -1).reshape(nt, heads * hd)

        K, V = st["k"].double().view(-1, nkv * hd), st["v"].double().view(-1, nkv * hd)
        at = _dev([place(b, s) for b, s in zip(st["seqs"].tolist(), st["slots"].tolist())], torch.int64)
        K[at], V[at] = finish(k, nkv, st["kw"]), v.double()
        return {"q": finish(q, nh, st["qw"]), "k": K.view(st["k"].shape), "v": V.view(st["v"].shape)}
    lens = st["lens"].tolist()
    K, V = st["k"].view(-1, nkv, hd), st["v"].view(-1, nkv, hd)
    if case["op"] == "attn":
        out = torch.zeros(case["batch"], nh * hd, dtype=torch.float64, device="cuda")
        weight = st["weight"].double() if case["weights"] else None
        for b, n in enumerate(lens):
            first = max(0, n - case["window"]) if case["window"] else 0
            if n == first:
                continue
            at = _dev([place(b, s) for s in range(first, n)], torch.int64)
            q = st["q"][b].double().view(nkv, nh // nkv, hd)
            s = torch.einsum("hgd,shd->hgs", q, K[at].double()) / math.sqrt(hd)
            p = torch.softmax(s, -1)
            out[b] = torch.einsum("hgs,shd->hgd", p, V[at].double()).reshape(-1)
            if weight is not None:
                weight[b, :, first:n] += p.sum(1)
        return {"out": out, "weight": weight} if case["weights"] else {"out": out}
    budget, recent = case["budget"], case["recent"]
    K, V = K.clone(), V.clone()
    weight, pos = st["weight"].cpu().numpy(), st["pos"].cpu().numpy()
    wo, po = weight.copy(), pos.copy()
    src, dst, heads = [], [], []
    for b, n in enumerate(lens):
        for h in range(nkv if n > budget else 0):
            w, t = weight[b, h, :n].tolist(), pos[b, h, :n].tolist()
            rank = sorted(range(n), key=lambda s: (t[s] < n - recent, 0.0 if t[s] >= n - recent else -w[s], s))
            kept = set(rank[:budget])
            holes = [s for s in range(budget) if s not in kept]
            movers = [s for s in range(budget, n) if s in kept]
            for i, j in zip(holes, movers):
                wo[b, h, i], po[b, h, i] = weight[b, h, j], pos[b, h, j]
                src.append(place(b, j))
                dst.append(place(b, i))
                heads.append(h)
    if src:
        src, dst, heads = (_dev(x, torch.int64) for x in (src, dst, heads))
        K[dst, heads], V[dst, heads] = K[src, heads], V[src, heads]
    shape = st["k"].shape
    return {"k": K.double().view(shape), "v": V.double().view(shape),
            "lens_out": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32),
            "weight_out": torch.from_numpy(wo).double(), "pos_out": torch.from_numpy(po)}
