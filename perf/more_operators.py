"""Cases, plain forms and exact values of rotary positions in their other forms and of attention of
many query rows over the paged cache.

Four operators, used one after the other when prompts that share a beginning are served:

  rope    rows of heads turned by their positions: half or interleaved pairs, all of a head or its
          first part, frequencies scaled for long contexts; or turned back, which is the gradient
          (qkv_rope_step)
  store   projected rows -> bias, optional q/k norms, that rotation, q out, k and v into the cache's
          pages (qkv_paged_store_rope_step)
  prompt  several new tokens of every sequence (a prompt, a part of one, drafted tokens) attend over
          its cached slots, each up to its own (qkv_prompt_attn_step)
  prefix  one new token of every sequence; the first slots of neighbouring sequences are the same
          pages and are read once for all of them (qkv_prefix_attn_step)

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
# Scalings of the frequencies: what a program that serves contexts beyond the trained length keeps
# (original length 32768), and the magnitude that goes with the ramp.
SCALING = {
    "none": dict(),
    "linear": dict(factor=4.0),
    "base": dict(factor=4.0),
    "ramp": dict(factor=4.0, orig_ctx=32768.0, low=1.0, high=32.0, magnitude=0.1 * math.log(4.0) + 1.0),
    "bands": dict(factor=8.0, orig_ctx=8192.0, low=1.0, high=4.0),
}


def listed():
    return [
        # the q and k heads of one 0.5B token: latency only
        dict(name="rope-0.5b-t1", op="rope", heads=16, hd=64, rot=64, layout="half", scaling="none", dtype="f32",
             tokens=1, far=32000, inverse=False),
        # the gradient of a 7B prompt's rotation, half of each head turned, in f16
        dict(name="rope-7b-t1641-back", op="rope", heads=32, hd=128, rot=64, layout="half", scaling="bands",
             dtype="f16", tokens=1641, far=32000, inverse=True),
        # q and k of a long 14B prompt in pairs of neighbours, far positions of a scaled context
        dict(name="rope-14b-t8191", op="rope", heads=48, hd=128, rot=128, layout="pairs", scaling="ramp", dtype="bf16",
             tokens=8191, far=120000, inverse=False),
        # the newest tokens of a 7B batch, pairs of neighbours in half of each head
        dict(name="store-7b-t32-pairs", op="store", nh=28, nkv=4, hd=128, rot=64, layout="pairs", scaling="none",
             kv="f16", page=16, mode="decode", tokens=32, y="f32", norm=False, far=32000),
        # a long 14B prompt with q/k norms, frequencies scaled for a long context
        dict(name="store-14b-t8191-ramp", op="store", nh=40, nkv=8, hd=128, rot=128, layout="half", scaling="ramp",
             kv="f16", page=64, mode="prompt", tokens=8191, y="bf16", norm=True, far=120000),
        # a short question on the 0.5B layer's own f32 cache: latency only
        dict(name="prompt-0.5b-b1-t17", op="prompt", nh=14, nkv=2, hd=64, kv="f32", page=16, batch=1, new=17, cached=0,
             ragged=False, window=0, out="f32"),
        # drafted tokens of an uneven 14B batch, checked in one call
        dict(name="prompt-14b-b32-t4", op="prompt", nh=40, nkv=8, hd=128, kv="f16", page=16, batch=32, new=4,
             cached=4099, ragged=True, window=0, out="f32"),
        # parts of four uneven 7B prompts behind what each has cached
        dict(name="prompt-7b-b4-t509", op="prompt", nh=28, nkv=4, hd=128, kv="f16", page=32, batch=4, new=509,
             cached=8192, ragged=True, window=0, out="bf16"),
        # a whole long 14B prompt
        dict(name="prompt-14b-b1-t8191", op="prompt", nh=40, nkv=8, hd=128, kv="f16", page=64, batch=1, new=8191,
             cached=0, ragged=False, window=0, out="bf16"),
        # four answers to one question on the 0.5B layer's own f32 cache: latency only
        dict(name="prefix-0.5b-b4-short", op="prefix", nh=14, nkv=2, hd=64, kv="f32", page=16, batch=4, groups=1,
             prefix=509, suffix=37, out="f32"),
        # a 14B batch under one instruction text
        dict(name="prefix-14b-b64", op="prefix", nh=40, nkv=8, hd=128, kv="f16", page=16, batch=64, groups=1,
             prefix=8192, suffix=1000, out="bf16"),
        # questions on two long documents on the 7B layout
        dict(name="prefix-7b-b96-long", op="prefix", nh=28, nkv=4, hd=128, kv="f16", page=64, batch=96, groups=2,
             prefix=32749, suffix=509, out="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _draw_rope(rng, hd):
    rot = rng.choice([hd, hd, hd // 2, hd // 4])
    return dict(rot=rot, layout=rng.choice(["half", "pairs"]), scaling=rng.choice(sorted(SCALING)),
                far=rng.choice([4000, 32000, 120000, 1000000]))


def draw(rng):
    op = rng.choice(["rope", "store", "prompt", "prompt", "prefix", "prefix"])
    nkv = rng.choice([1, 2, 4, 5, 8])
    hd = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
    if op == "rope":
        heads = _log(rng, 1, 64)
        return dict(op=op, heads=heads, hd=hd, dtype=rng.choice(["f32", "bf16", "f16"]),
                    tokens=_log(rng, 1, min(40000, 8191 * 6144 // (heads * hd))), inverse=rng.random() < 0.4,
                    **_draw_rope(rng, hd))
    c = dict(op=op, nh=nkv * rng.choice([1, 2, 4, 5, 7, 8, 12]), nkv=nkv, hd=hd, kv=rng.choice(["f16", "f16", "f16", "f32"]),
             page=rng.choice([1, 8, 16, 17, 32, 64, 128, 256]))
    if op == "store":
        c.update(mode=rng.choice(["decode", "prompt"]), y=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.6,
                 **_draw_rope(rng, hd))
        most = 8191 * 7168 // ((c["nh"] + 2 * nkv) * hd)
        c["tokens"] = _log(rng, 1, min(256 if c["mode"] == "decode" else 8191, most))
        return c
    c["out"] = rng.choice(["f32", "bf16"])
    # no more cached values than in 33000 slots of the largest layout, in all sequences together
    room = (1 << 25) // (nkv * hd)
    if op == "prompt":
        c["batch"] = _log(rng, 1, 64)
        c["new"] = _log(rng, 1, max(1, min(4096, room // c["batch"])))
        c["cached"] = rng.choice([0, _log(rng, 1, max(1, min(32768, room // c["batch"])))])
        # no more scores than a quarter of the largest listed case's
        most = 8191 * 8191 * 40 // 4 // (c["nh"] * c["batch"] * (c["new"] + c["cached"]))
        c["new"] = max(1, min(c["new"], most))
        c["ragged"] = rng.random() < 0.7
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        return c
    c["batch"] = _log(rng, 1, 128)
    c["groups"] = rng.choice([1, 1, 2, 3]) if c["batch"] >= 3 else 1
    c["prefix"] = _log(rng, 1, min(32768, room // c["groups"]))
    c["suffix"] = _log(rng, 1, max(1, min(2048, room // c["batch"])))
    return c


# ---------------------------------------------------------------- inputs

def _rope_config(case):
    return dict(hd=case["hd"], rot=case["rot"], scaling=case["scaling"], **SCALING[case["scaling"]])


def _freqs(c):
    """Angle of each pair for one step of position, in 64 bits."""
    rot, f = c["rot"], c.get("factor", 1.0)
    theta = THETA * f ** (rot / (rot - 2.0)) if c["scaling"] == "base" else THETA
    freq = [theta ** (-2.0 * d / rot) for d in range(rot // 2)]
    if c["scaling"] == "linear":
        freq = [x / f for x in freq]
    elif c["scaling"] == "ramp":
        # pair index at which a turn count over the original context is reached
        at = lambda turns: rot * math.log(c["orig_ctx"] / (2 * math.pi * turns)) / (2 * math.log(THETA))  # noqa: E731
        lo, hi = max(0.0, float(math.floor(at(c["high"])))), min(rot - 1.0, float(math.ceil(at(c["low"]))))
        for d, x in enumerate(freq):
            g = min(1.0, max(0.0, (d - lo) / max(hi - lo, 0.001)))
            freq[d] = x / f * g + x * (1.0 - g)
    elif c["scaling"] == "bands":
        for d, x in enumerate(freq):
            turns = c["orig_ctx"] * x / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - c["low"]) / (c["high"] - c["low"])))
            freq[d] = (1.0 - g) * x / f + g * x
    return freq


def _cache(case, gen, counts, shared=None):
    """Pools whose rows all hold numbers, pages scattered; sequence b has counts[b] pages of its own, behind the first
    n pages of another where shared[b] is (that sequence, n)."""
    ps, nkv, hd = case["page"], case["nkv"], case["hd"]
    total = sum(counts) + 3
    ids = iter(torch.randperm(total, generator=gen, device="cuda").tolist())
    rows = []
    for b, n in enumerate(counts):
        lead, common = shared[b] if shared else (0, 0)
        rows.append((rows[lead][:common] if common else []) + [next(ids) for _ in range(n)])
    most = max(1, max(len(row) for row in rows))
    table = torch.tensor([row + [0] * (most - len(row)) for row in rows], dtype=torch.int32, device="cuda")
    pools = [torch.empty(total, ps, nkv * hd, dtype=DT[case["kv"]], device="cuda") for _ in range(2)]
    for p in pools:
        p.normal_(generator=gen)
    return dict(k=pools[0], v=pools[1], table=table, cap=most * ps)


def _new_tokens(case):
    """How many new tokens the sequences have: evenly spread from few to the most, or the most each."""
    B, n = case["batch"], case["new"]
    return [n * (i + 1) // B if case["ragged"] else n for i in range(B)]


def _dev(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    hd = case["hd"]
    if case["op"] == "rope":
        nt = case["tokens"]
        first = r.randint(0, case["far"])
        x = rand(nt, case["heads"] * hd).to(DT[case["dtype"]])
        return dict(x=x, out=torch.empty_like(x), pos=_dev([first + t for t in range(nt)]),
                    freq=_dev(_freqs(_rope_config(case)), torch.float64))
    nh, nkv, ps = case["nh"], case["nkv"], case["page"]
    if case["op"] == "store":
        nt = case["tokens"]
        if case["mode"] == "decode":  # token t is the newest of sequence t
            per = -(-max(ps, 64) // ps)
            pos = [r.randint(0, case["far"]) for _ in range(nt)]
            seqs, slots = list(range(nt)), [r.randrange(per * ps) for _ in range(nt)]
            st = _cache(case, gen, [per] * nt)
        else:  # one sequence's prompt behind what it has cached, at far positions
            first, at = r.randint(0, 2000), r.randint(0, case["far"])
            pos, seqs, slots = [at + t for t in range(nt)], [0] * nt, [first + t for t in range(nt)]
            st = _cache(case, gen, [-(-(2000 + nt) // ps)])
        R = (nh + 2 * nkv) * hd
        st["y"] = rand(nt, R).to(DT[case["y"]])
        st["bias"] = 0.1 * rand(R)
        st["qw"], st["kw"] = (1 + 0.1 * rand(hd), 1 + 0.1 * rand(hd)) if case["norm"] else (None, None)
        st["pos"], st["seqs"], st["slots"] = _dev(pos), _dev(seqs), _dev(slots)
        st["q"] = torch.empty(nt, nh * hd, device="cuda")
        st["freq"] = _dev(_freqs(_rope_config(case)), torch.float64)
        return st
    B = case["batch"]
    if case["op"] == "prompt":
        new = _new_tokens(case)
        r.shuffle(new)
        cached = [r.randint(0, case["cached"]) if case["ragged"] else case["cached"] for _ in range(B)]
        cached[r.randrange(B)] = case["cached"]
        lens = [n + c for n, c in zip(new, cached)]
        st = _cache(case, gen, [-(-n // ps) for n in lens])
        first = [0]
        for n in new:
            first.append(first[-1] + n)
        st.update(first=_dev(first), lens=_dev(lens), host=(first, lens), nt=first[-1])
        rows = first[-1]
    else:
        # neighbouring sequences share the pages of a prefix that ends on a page's border; the rest is each one's own
        edge = [r.randint(0, B - 1) for _ in range(case["groups"] - 1)]
        share, counts, shared, lens, prefix = [], [], [], [], []
        for b in range(B):
            lead = b if b == 0 or b in edge else share[-1]
            suffix = r.randint(1, case["suffix"])
            if lead == b:
                common = (case["prefix"] if b == 0 else r.randint(1, case["prefix"])) // ps
                counts.append(common + -(-suffix // ps))
                shared.append((b, 0))
            else:
                common = prefix[lead] // ps
                counts.append(-(-suffix // ps))
                shared.append((lead, common))
            share.append(lead)
            prefix.append(common * ps)
            lens.append(prefix[-1] + suffix)
        st = _cache(case, gen, counts, shared)
        st.update(lens=_dev(lens), share=_dev(share), prefix=_dev(prefix), host=(lens, share, prefix))
        rows = B
    st["q"] = 2.0 * rand(rows, nh * hd)
    st["out"] = torch.empty(rows, nh * hd, dtype=DT[case["out"]], device="cuda")
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    st["mag"] = SCALING[case["scaling"]].get("magnitude", 1.0) if "scaling" in case else 1.0
    if own:
        import qkv_rope_kv_gb300 as Q
        st["Q"] = Q
        if "rot" in case:
            kind = {"none": Q.QKV_ROPE_SCALE_NONE, "linear": Q.QKV_ROPE_SCALE_LINEAR, "base": Q.QKV_ROPE_SCALE_BASE,
                    "ramp": Q.QKV_ROPE_SCALE_RAMP, "bands": Q.QKV_ROPE_SCALE_BANDS}[case["scaling"]]
            layout = {"half": Q.QKV_ROPE_NEOX, "pairs": Q.QKV_ROPE_INTERLEAVED}[case["layout"]]
            st["rope"] = Q.qkv_rope_create(case["hd"], THETA, rot_dim=case["rot"], layout=layout, scaling=kind,
                                           **SCALING[case["scaling"]])
        if case["op"] != "rope":
            kv = {"f32": Q.QKV_F32, "f16": Q.QKV_F16}[case["kv"]]
            plan = Q.qkv_plan_create(case["nh"] * case["hd"], case["nh"], case["nkv"], case["hd"], THETA, st["cap"],
                                     w_dtype=Q.QKV_BF16, kv_dtype=kv)
            cache = Q.PagedKv(plan, st["k"], st["v"], st["table"])
            st.update(plan=plan, cache=cache)
            if case["op"] != "store":
                need = (Q.qkv_prompt_attn_workspace_bytes(plan, cache, st["nt"]) if case["op"] == "prompt"
                        else Q.qkv_prefix_attn_workspace_bytes(plan, cache))
                st["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return {"rope": _rope, "store": _store, "prompt": _prompt, "prefix": _prefix}[st["case"]["op"]](st)


def _turn(st, x, inverse=False):
    """x [nt, heads, hd] (f32) turned by its tokens' positions."""
    c, rot = st["case"], st["case"]["rot"]
    angle = st["pos"].double()[:, None] * st["freq"]
    cos, sin = (st["mag"] * angle.cos()).float()[:, None], (st["mag"] * angle.sin()).float()[:, None]
    if inverse:
        sin = -sin
    head, rest = x[..., :rot], x[..., rot:]
    if c["layout"] == "half":
        x0, x1 = head[..., :rot // 2], head[..., rot // 2:]
        return torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos, rest], -1)
    x0, x1 = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2), rest], -1)


def _rope(st):
    c = st["case"]
    if own:
        st["Q"].qkv_rope_step(st["rope"], st["x"], st["pos"], st["out"], inverse=c["inverse"])
    else:
        x = st["x"].float().view(c["tokens"], c["heads"], c["hd"])
        st["out"].copy_(_turn(st, x, c["inverse"]).reshape(c["tokens"], -1))
    return st["out"]


def _rows(st, b, slots):
    """Row numbers in the pools, seen as [pages * page, nkt], of `slots` of sequence (or sequences) b."""
    ps = st["case"]["page"]
    slots = slots.long()
    return st["table"].long()[b, slots // ps] * ps + slots % ps


def _store(st):
    c = st["case"]
    if own:
        st["Q"].qkv_paged_store_rope_step(st["plan"], st["cache"], st["rope"], st["y"], st["bias"], st["qw"], st["kw"],
                                          EPS, st["pos"], st["seqs"], st["slots"], st["q"])
        return {"q": st["q"], "k": st["k"], "v": st["v"]}
    nh, nkv, hd, nt = c["nh"], c["nkv"], c["hd"], c["tokens"]
    z = (st["y"].float() + st["bias"]).view(nt, nh + 2 * nkv, hd)
    qk, v = z[:, :nh + nkv], z[:, nh + nkv:]
    if c["norm"]:
        w = torch.cat([st["qw"].expand(nh, hd), st["kw"].expand(nkv, hd)])
        qk = qk / torch.sqrt(qk.square().mean(-1, keepdim=True) + EPS) * w
    qk = _turn(st, qk)
    st["q"].copy_(qk[:, :nh].reshape(nt, -1))
    rows = _rows(st, st["seqs"].long(), st["slots"])
    st["k"].view(-1, nkv * hd)[rows] = qk[:, nh:].reshape(nt, -1).to(st["k"].dtype)
    st["v"].view(-1, nkv * hd)[rows] = v.reshape(nt, -1).to(st["v"].dtype)
    return {"q": st["q"], "k": st["k"], "v": st["v"]}


def _softmax_sum(s, seen, v):
    """softmax over the seen scores, times v: all in f32; a row that sees nothing gives zeros."""
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, 1.0, total)


def _prompt(st):
    c = st["case"]
    nh, nkv, hd = c["nh"], c["nkv"], c["hd"]
    scale = hd ** -0.5
    if own:
        st["Q"].qkv_prompt_attn_step(st["plan"], st["cache"], st["q"], st["first"], st["lens"], scale, st["out"],
                                     st["ws"], window=c["window"])
        return st["out"]
    first, lens = st["host"]
    kp, vp = st["k"].view(-1, nkv, hd), st["v"].view(-1, nkv, hd)
    G = nh // nkv
    for b, n in enumerate(lens):
        new = first[b + 1] - first[b]
        if new == 0:
            continue
        slots = torch.arange(n, device="cuda")
        rows = _rows(st, b, slots)
        end = n - new + torch.arange(new, device="cuda")[:, None]  # the row's own slot
        seen = slots <= end
        if c["window"]:
            seen = seen & (slots > end - c["window"])
        q = (st["q"][first[b]:first[b + 1]] * scale).view(new, nkv, G, hd)
        out = torch.empty(new, nkv, G, hd, device="cuda")
        for h in range(nkv):
            k, v = kp[rows, h].float(), vp[rows, h].float()
            s = (q[:, h].reshape(new * G, hd) @ k.t()).view(new, G, n)
            out[:, h] = _softmax_sum(s, seen[:, None], v)
        st["out"][first[b]:first[b + 1]] = out.view(new, nh * hd).to(st["out"].dtype)
    return st["out"]


def _prefix(st):
    c = st["case"]
    nh, nkv, hd = c["nh"], c["nkv"], c["hd"]
    scale = hd ** -0.5
    if own:
        st["Q"].qkv_prefix_attn_step(st["plan"], st["cache"], st["q"], st["lens"], st["share"], st["prefix"], scale,
                                     st["out"], st["ws"])
        return st["out"]
    lens, share, prefix = st["host"]
    kp, vp = st["k"].view(-1, nkv, hd), st["v"].view(-1, nkv, hd)
    G = nh // nkv
    q = (st["q"] * scale).view(-1, nkv, G, hd)
    b = 0
    while b < c["batch"]:
        e = b
        while e < c["batch"] and share[e] == share[b]:
            e += 1
        # the group's prefix once for all its rows, the rest sequence by sequence in one padded product
        P, most = prefix[b], max(lens[i] - prefix[i] for i in range(b, e))
        rows = _rows(st, share[b], torch.arange(P, device="cuda"))
        own_slots = torch.arange(most, device="cuda")
        n = st["lens"][b:e].long() - P
        own_rows = _rows(st, torch.arange(b, e, device="cuda")[:, None],
                         torch.minimum(P + own_slots[None], st["lens"][b:e].long()[:, None] - 1))
        k, v = kp[rows].float().permute(1, 2, 0), vp[rows].float().transpose(0, 1)          # [nkv, hd, P], [nkv, P, hd]
        ko, vo = kp[own_rows].float().permute(0, 2, 3, 1), vp[own_rows].float().transpose(1, 2)
        x = q[b:e].permute(1, 0, 2, 3).reshape(nkv, (e - b) * G, hd)
        s0 = (x @ k).view(nkv, e - b, G, P).transpose(0, 1)
        s1 = torch.where((own_slots < n[:, None])[:, None, None], q[b:e] @ ko, -math.inf)
        m = torch.maximum(s0.amax(-1, keepdim=True) if P else s1.amax(-1, keepdim=True), s1.amax(-1, keepdim=True))
        p0, p1 = torch.exp(s0 - m), torch.exp(s1 - m)
        o0 = (p0.transpose(0, 1).reshape(nkv, (e - b) * G, P) @ v).view(nkv, e - b, G, hd).transpose(0, 1)
        out = (o0 + p1 @ vo) / (p0.sum(-1, keepdim=True) + p1.sum(-1, keepdim=True))
        st["out"][b:e] = out.reshape(e - b, nh * hd).to(st["out"].dtype)
        b = e
    return st["out"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    hd = case["hd"]
    if case["op"] == "rope":
        nt, n = case["tokens"], case["tokens"] * case["heads"] * hd
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 4 * nt, "flops": nt * case["rot"] * (3 * case["heads"] + 4)}
    nh, nkv, e = case["nh"], case["nkv"], SIZE[case["kv"]]
    if case["op"] == "store":
        nt, R = case["tokens"], (nh + 2 * nkv) * hd
        return {"bytes": nt * (R * SIZE[case["y"]] + 4 * nh * hd + 2 * nkv * hd * e + 12) + 4 * R,
                "flops": nt * R * 8}
    row = nh * hd * (4 + SIZE[case["out"]])
    slot = 2 * nkv * hd * e
    B = case["batch"]
    if case["op"] == "prompt":
        w, nt, scores, slots = case["window"], 0, 0, 0
        for i, n in enumerate(_new_tokens(case)):
            c = case["cached"] / 2 if case["ragged"] and i else case["cached"]  # ragged: one full, the others uniform
            nt += n
            scores += sum(min(c + t + 1, w) if w else c + t + 1 for t in range(n))
            slots += (min(n + c, w + n - 1) if w else n + c) if n else 0
        return {"bytes": nt * row + slots * slot + 4 * slots / case["page"], "flops": 4 * scores * nh * hd}
    # the first group's prefix is full, the others' uniform up to it; suffixes uniform up to the longest
    shared = case["prefix"] * (1 + (case["groups"] - 1) / 2)
    suffix = (case["suffix"] + 1) / 2
    mean = shared / case["groups"] + suffix
    return {"bytes": B * row + (shared + B * suffix) * slot + 4 * (shared + B * suffix) / case["page"],
            "flops": 4 * B * mean * nh * hd}


# ---------------------------------------------------------------- the definition in 64 bits

def _turned(case, st, x):
    """x [nt, heads, hd] in 64 bits, as complex numbers times e^(i angle)."""
    rot, mag = case["rot"], SCALING[case["scaling"]].get("magnitude", 1.0)
    freq = torch.tensor(_freqs(_rope_config(case)), dtype=torch.float64, device="cuda")
    angle = torch.outer(st["pos"].double(), freq)
    by = torch.polar(torch.full_like(angle, mag), -angle if case.get("inverse") else angle)[:, None]
    y = x.clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * by
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * by
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    return y


def _attend(q, K, V, lo, hi, scale):
    """q [rows, G, hd], K and V [n, hd] in 64 bits; row i sees slots lo[i] .. hi[i] - 1."""
    out = torch.zeros_like(q)
    n = K.shape[0]
    step = max(1, (1 << 26) // max(1, n * q.shape[1]))
    at = torch.arange(n, device="cuda")
    for i in range(0, q.shape[0], step):
        s = torch.einsum("rgd,nd->rgn", q[i:i + step], K) * scale
        hidden = (at < lo[i:i + step, None]) | (at >= hi[i:i + step, None])
        s.masked_fill_(hidden[:, None], -math.inf)
        p = torch.nan_to_num(torch.softmax(s, -1))  # a row that sees nothing
        out[i:i + step] = torch.einsum("rgn,nd->rgd", p, V)
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    hd = case["hd"]
    if case["op"] == "rope":
        x = st["x"].double().view(case["tokens"], case["heads"], hd)
        return _turned(case, st, x).reshape(case["tokens"], -1)
    nh, nkv, ps = case["nh"], case["nkv"], case["page"]
    table = st["table"].cpu()
    if case["op"] == "store":
        nt = case["tokens"]
        z = st["y"].double() + st["bias"].double()
        q, k, v = z.split([nh * hd, nkv * hd, nkv * hd], 1)

        def finish(x, heads, w):
            x = x.reshape(nt, heads, hd)
            if case["norm"]:
                x = x * w.double() * (x.pow(2).sum(-1, keepdim=True) / hd + EPS).pow(-0.5)
            return _turned(case, st, x).reshape(nt, heads * hd)

        K, V = st["k"].double().view(-1, nkv * hd), st["v"].double().view(-1, nkv * hd)
        at = _dev([int(table[b, s // ps]) * ps + s % ps for b, s in zip(st["seqs"].tolist(), st["slots"].tolist())],
                  torch.int64)
        K[at], V[at] = finish(k, nkv, st["kw"]), v.double()
        return {"q": finish(q, nh, st["qw"]), "k": K.view(st["k"].shape), "v": V.view(st["v"].shape)}
    G = nh // nkv
    K, V = st["k"].view(-1, nkv, hd), st["v"].view(-1, nkv, hd)
    q = st["q"].double().view(-1, nkv, G, hd)
    out = torch.zeros_like(q)
    lens = st["lens"].tolist()
    first = st["first"].tolist() if case["op"] == "prompt" else list(range(case["batch"] + 1))
    for b, n in enumerate(lens):
        a, e = first[b], first[b + 1]
        if e == a or n == 0:
            continue
        s = torch.arange(n)
        at = (table[b].long()[s // ps] * ps + s % ps).cuda()
        hi = torch.arange(n - (e - a) + 1, n + 1, device="cuda")
        lo = (hi - case["window"]).clamp(min=0) if case.get("window") else torch.zeros_like(hi)
        for h in range(nkv):
            out[a:e, h] = _attend(q[a:e, h], K[at, h].double(), V[at, h].double(), lo, hi, 1.0 / math.sqrt(hd))
    return out.view(-1, nh * hd)
