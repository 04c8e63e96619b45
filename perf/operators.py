"""What is measured of the operators on a 4-bit KV cache: writing it, attention over it
for single tokens and for chunks of a prompt, and eviction by accumulated attention
weight.

A cache row is one token's key or value of one KV head.  It is held in groups of 32
dims; a group is a bf16 offset `lo`, a bf16 step `s` and one code of 0..15 for each dim:

    lo   = the largest bf16 <= min(x)          s = the smallest bf16 >= (max(x) - lo) / 15
    code = round((x - lo) / s), ties to even   value = lo + s * code    (s = 0: value = lo)

Attention reads these values.  Accumulated weights: weight[b][h][slot] grows by the
softmax probabilities that the query heads of KV head h give the slot's token.  Eviction
keeps the first tokens, the newest ones, and of the others those of the largest weights
(ties: the lower slot), and moves the kept rows that sit past the budget into the slots
that became free (the j-th such row, by slot, into the j-th free slot).

Every function here takes plain values or what prepare() made.  With `own` false run()
computes in elementary torch operations; with `own` true it makes the library's calls.
"""
import math

import torch

own = False

GROUP = 32
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------
def _case(name, op, dtype, B, Hq, Hkv, d, L, ragged, n=1, acc=0, budget=0, first=0, recent=0):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "d": d,
            "L": L, "ragged": ragged, "n": n, "acc": acc, "budget": budget, "first": first,
            "recent": recent}


def listed():
    return [
        # a short prompt of a small fp32 model, three sequences of odd lengths
        _case("write f32 777x3", "write", "f32", 3, 4, 2, 64, 777, True),
        # a whole long prompt of one sequence goes into the cache
        _case("write bf16 131072", "write", "bf16", 1, 32, 8, 128, 131072, False),
        # the first tokens of an answer: the smallest call
        _case("decode bf16 37", "decode", "bf16", 1, 32, 8, 128, 37, False),
        # a serving batch of short fp32 sequences, weights accumulated for a later eviction
        _case("decode f32 16x3999 weights", "decode", "f32", 16, 16, 8, 64, 3999, True, acc=1),
        # one long sequence, latency bound by the cache read; weights accumulated
        _case("decode bf16 131072 weights", "decode", "bf16", 1, 32, 8, 128, 131072, False, acc=1),
        # the benchmark's own decode shape: four sequences of 524288
        _case("decode bf16 4x524288", "decode", "bf16", 4, 32, 8, 128, 524288, False),
        # a few drafted tokens of eight sequences are scored at once
        _case("chunk bf16 5x8 at 9001", "chunk", "bf16", 8, 32, 8, 128, 9001, True, n=5),
        # an fp32 chunk whose newest rows feed the weights
        _case("chunk f32 100x2 at 2500 weights", "chunk", "f32", 2, 8, 2, 64, 2500, True, n=100,
              acc=33),
        # a chunk of a long prompt
        _case("chunk bf16 512 at 32768", "chunk", "bf16", 1, 32, 8, 128, 32768, False, n=512),
        # the last chunk of a prompt that fits one call, its newest rows feed the weights
        _case("chunk bf16 2048 at 16384 weights", "chunk", "bf16", 1, 32, 8, 128, 16384, False,
              n=2048, acc=32),
        # a decode step of a bounded cache: one token comes, one goes
        _case("evict bf16 1 of 4096x4", "evict", "bf16", 4, 32, 8, 128, 4096, False, n=1,
              budget=4096, first=4, recent=256),
        # a chunk comes and the cache shrinks back to its bound
        _case("evict f32 2048 of 8192x2", "evict", "f32", 2, 16, 4, 128, 8192, True, n=2048,
              budget=8192, first=16, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "decode", "chunk", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 16)
    c = dict(op=op, dtype=dtype, B=B, Hq=G * Hkv, Hkv=Hkv, d=d, ragged=rng.random() < 0.5, n=1,
             acc=0, budget=0, first=0, recent=0)
    rows = 1 << 20                       # tokens x KV heads of one cache
    if op == "write":
        c["L"] = _log(rng, 16, rows // (B * Hkv))
    elif op == "decode":
        c["L"] = _log(rng, 1, 4 * rows // (B * Hkv))
        c["acc"] = rng.choice([0, 1])
    elif op == "chunk":
        c["n"] = _log(rng, 2, 1024)
        most = min(rows // (B * Hkv), (1 << 29) // (B * Hkv * G * c["n"]))
        c["L"] = c["n"] + _log(rng, 1, max(2, most))
        c["acc"] = rng.choice([0, 0, min(c["n"], rng.randint(1, 64))])
    else:
        c["budget"] = _log(rng, 64, max(65, rows // (4 * B * Hkv)))
        c["n"] = _log(rng, 1, c["budget"])
        c["L"] = c["budget"]
        c["first"] = rng.randint(0, 16)
        c["recent"] = rng.randint(0, c["budget"] // 2)
    return c


def _lengths(c):
    """The sequences' lengths; ragged ones fall by 37/64 of L over the batch."""
    B, L, least = c["B"], c["L"], c["n"] if c["op"] == "chunk" else 1
    return [max(least, L - (37 * L * b) // (64 * B)) if c["ragged"] else L for b in range(B)]


def _capacity(c):
    return c["L"] + (c["n"] if c["op"] == "evict" else 0) + 5


# ---------------------------------------------------------------------------------
# inputs (from the seed alone)
# ---------------------------------------------------------------------------------
def _kv_inputs(c, seed):
    """K and V of one sequence at a time: [Hkv][L][d].  Keys have channels of unequal
    size and offset, as keys of trained models have; values are N(0, 1)."""
    g = torch.Generator(device=DEV).manual_seed(1_000_003 * seed + 1)
    H, L, d, dt = c["Hkv"], c["L"], c["d"], _DT[c["dtype"]]
    size = torch.exp(0.4 * torch.randn(H, 1, d, generator=g, device=DEV))
    off = 0.7 * torch.randn(H, 1, d, generator=g, device=DEV)
    for _ in range(c["B"]):
        k = torch.randn(H, L, d, generator=g, device=DEV).mul_(size).add_(off).to(dt)
        v = torch.randn(H, L, d, generator=g, device=DEV).to(dt)
        yield k, v


def _other_inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(1_000_003 * seed + 2)
    dt = _DT[c["dtype"]]
    x = {}
    if c["op"] in ("decode", "chunk"):
        x["q"] = torch.randn(c["B"], c["n"], c["Hq"], c["d"], generator=g, device=DEV).to(dt)
    if c["op"] == "evict":
        shape = (c["B"], c["Hkv"], c["n"], c["d"])
        x["k_new"] = torch.randn(shape, generator=g, device=DEV).to(dt)
        x["v_new"] = torch.randn(shape, generator=g, device=DEV).to(dt)
        # weights as attention leaves them: a few large, many small, some equal
        w = -torch.log(torch.rand(c["B"], c["Hkv"], c["L"], generator=g, device=DEV))
        there = torch.arange(c["L"], device=DEV) < torch.tensor(_lengths(c), device=DEV)[:, None]
        x["w_in"] = torch.where((w > 0.05) & there.unsqueeze(1), w, 0.0)
    return x


# ---------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------
def _quantize(x):
    """codes uint8 [.., d/2] (dim 2j low, dim 2j+1 high), s and lo bf16 [.., d/32]."""
    g = x.unflatten(-1, (x.shape[-1] // GROUP, GROUP))
    bits = g.amin(-1).float().view(torch.int32)
    cut = bits & -65536
    lo = torch.where((bits < 0) & (bits != cut), cut + 65536, cut).view(torch.float32)
    want = (g.amax(-1).double() - lo.double()) / 15
    s = want.float()
    s = torch.where(s.double() < want, (s.view(torch.int32) + 1).view(torch.float32), s)
    bits = s.view(torch.int32)
    cut = bits & -65536
    s = torch.where(bits != cut, cut + 65536, cut).view(torch.float32)
    t = (g.double() - lo.double().unsqueeze(-1)) / torch.where(s > 0, s, 1.0).double().unsqueeze(-1)
    code = t.round_().clamp_(0, 15).to(torch.uint8).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)), s.bfloat16(), lo.bfloat16()


def _values(code, s, lo):
    """fp32 values of a cache [.., d/2] codes with [.., d/32] steps and offsets."""
    c = torch.stack((code & 15, code >> 4), -1).flatten(-2).float()
    c = c.unflatten(-1, (s.shape[-1], GROUP))
    return c.mul_(s.float().unsqueeze(-1)).add_(lo.float().unsqueeze(-1)).flatten(-2)


def _plain_cache(c, seed):
    B, H, d, cap = c["B"], c["Hkv"], c["d"], _capacity(c)
    st = {"codes": [], "s": [], "lo": []}
    for _ in range(2):
        st["codes"].append(torch.zeros(B, H, cap, d // 2, dtype=torch.uint8, device=DEV))
        st["s"].append(torch.zeros(B, H, cap, d // GROUP, dtype=torch.bfloat16, device=DEV))
        st["lo"].append(torch.zeros(B, H, cap, d // GROUP, dtype=torch.bfloat16, device=DEV))
    for b, kv in enumerate(_kv_inputs(c, seed)):
        for i, x in enumerate(kv):
            for h in range(H):
                code, s, lo = _quantize(x[h])
                st["codes"][i][b, h, :c["L"]] = code
                st["s"][i][b, h, :c["L"]] = s
                st["lo"][i][b, h, :c["L"]] = lo
    st["len"] = torch.tensor(_lengths(c), device=DEV)
    st["pos"] = torch.arange(cap, device=DEV, dtype=torch.int32).repeat(B, H, 1)
    st["seen"] = st["len"].clone()
    st["w"] = torch.zeros(B, H, cap, device=DEV)
    return st


def _run_write(st):
    c, slot = st["case"], torch.arange(st["case"]["L"], device=DEV)
    there = (slot < st["len"].unsqueeze(1))[:, None, :, None]
    out = {}
    for name in ("k", "v"):
        v = _values(*_quantize(st[name]))
        out[name] = torch.where(there, v, torch.zeros((), device=DEV)).to(_DT[c["dtype"]])
    return out


def _run_attend(st):
    c = st["case"]
    B, H, d, n, L = c["B"], c["Hkv"], c["d"], c["n"], c["L"]
    G = c["Hq"] // H
    k, v = (_values(st["codes"][i][:, :, :L], st["s"][i][:, :, :L], st["lo"][i][:, :, :L])
            for i in range(2))
    q = st["q"].float().view(B, n, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, d)
    s = (q @ k.transpose(-1, -2)).view(B, H, n, G, L).mul_(d ** -0.5)
    # row i of a sequence sits at position seen - n + i and sees the slots up to there
    at = st["seen"].unsqueeze(1) - n + torch.arange(n, device=DEV)
    sees = st["pos"][:, :, None, :L] <= at[:, None, :, None]
    sees = sees & (torch.arange(L, device=DEV) < st["len"].unsqueeze(1))[:, None, None, :]
    s = s.masked_fill_(~sees.unsqueeze(3), -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True))
    o = (p.view(B, H, n * G, L) @ v).view(B, H, n, G, d).permute(0, 2, 1, 3, 4)
    out = {"out": o.reshape(B, n, H * G, d).to(_DT[c["dtype"]])}
    if c["acc"]:
        rows = c["acc"] if c["op"] == "chunk" else 1
        st["w"][:, :, :L] += p[:, :, n - rows:].sum((2, 3))
        out["weights"] = st["w"][:, :, :L]
    return out


def _run_evict(st):
    c = st["case"]
    B, H, n, keep = c["B"], c["Hkv"], c["n"], c["budget"]
    # the new rows go behind the cached ones
    at = (st["len"].unsqueeze(1) + torch.arange(n, device=DEV))[:, None, :].expand(B, H, n)
    for i, name in enumerate(("k_new", "v_new")):
        for part, x in zip(("codes", "s", "lo"), _quantize(st[name])):
            st[part][i].scatter_(2, at.unsqueeze(-1).expand(*x.shape), x)
    pos = (st["seen"].unsqueeze(1) + torch.arange(n, device=DEV)).to(torch.int32)
    st["pos"].scatter_(2, at, pos[:, None, :].expand(B, H, n))
    st["w"].scatter_(2, at, torch.zeros(B, H, n, device=DEV))
    st["len"] += n
    st["seen"] += n
    # rank: the protected ones, then by weight, ties to the lower slot
    L = c["L"] + n
    slot = torch.arange(L, device=DEV)
    there = (slot < st["len"].unsqueeze(1)).unsqueeze(1)
    p = st["pos"][:, :, :L]
    safe = (p < c["first"]) | (p >= (st["seen"] - c["recent"])[:, None, None])
    key = torch.where(safe, math.inf, st["w"][:, :, :L])
    key = torch.where(there, key, -1.0)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros(B, H, L, dtype=torch.bool, device=DEV)
    kept.scatter_(2, order[:, :, :keep], True)
    kept &= there
    free = (there & ~kept & (slot < keep)).nonzero(as_tuple=True)
    come = (kept & (slot >= keep)).nonzero(as_tuple=True)
    for t in [*st["codes"], *st["s"], *st["lo"], st["pos"], st["w"]]:
        t[free] = t[come]
    st["len"].clamp_(max=keep)
    there = slot[:keep] < st["len"].unsqueeze(1)
    out = {}
    for i, name in enumerate(("k", "v")):
        v = _values(st["codes"][i][:, :, :keep], st["s"][i][:, :, :keep], st["lo"][i][:, :, :keep])
        out[name] = torch.where(there[:, None, :, None], v, 0.0).to(_DT[c["dtype"]])
    out["positions"] = torch.where(there.unsqueeze(1), st["pos"][:, :, :keep], 0)
    out["weights"] = torch.where(there.unsqueeze(1), st["w"][:, :, :keep], 0.0)
    out["lengths"] = st["len"].clone()
    return out


# ---------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------
def _own_cache(c, seed):
    import long_context_recsa_b200.recsa as R
    cfg = R.Config(head_dim=c["d"], n_q_heads=c["Hq"], n_kv_heads=c["Hkv"], dtype=c["dtype"])
    return R.RecsaKV4(cfg, _capacity(c), c["B"], max_queries=c["B"] * c["n"])


def _own_prepare(c, seed):
    st = {"kv4": _own_cache(c, seed)}
    if c["op"] == "write":
        return st
    k = torch.empty(c["B"], c["Hkv"], c["L"], c["d"], dtype=_DT[c["dtype"]], device=DEV)
    v = torch.empty_like(k)
    for b, (kb, vb) in enumerate(_kv_inputs(c, seed)):
        k[b], v[b] = kb, vb
    st["kv4"].recsa_kv4_build(k, v, _lengths(c))
    return st


def _own_run(st):
    c, kv4 = st["case"], st["kv4"]
    if c["op"] == "write":
        kv4.recsa_kv4_build(st["k"], st["v"], _lengths(c))
        k, v = kv4.read(0, c["L"])
        return {"k": k, "v": v}
    if c["op"] == "decode":
        out = {"out": kv4.decode(st["q"][:, 0], accumulate=bool(c["acc"])).unsqueeze(1)}
    elif c["op"] == "chunk":
        out = {"out": kv4.prefill(st["q"], accumulate_rows=c["acc"])}
    else:
        kv4.recsa_kv4_append(st["k_new"], st["v_new"])
        kv4.recsa_kv4_evict(c["budget"], c["first"], c["recent"])
        k, v = kv4.read(0, c["budget"])
        return {"k": k, "v": v, "positions": kv4.positions()[:, :, :c["budget"]],
                "weights": kv4.weights()[:, :, :c["budget"]], "lengths": kv4.lengths()}
    if c["acc"]:
        out["weights"] = kv4.weights()[:, :, :c["L"]]
    return out


# ---------------------------------------------------------------------------------
# what the tools call
# ---------------------------------------------------------------------------------
def prepare(case, seed):
    c = dict(case)
    if own:
        st = _own_prepare(c, seed)
    elif c["op"] == "write":
        st = {"len": torch.tensor(_lengths(c), device=DEV)}
    else:
        st = _plain_cache(c, seed)
    st["case"] = c
    if c["op"] == "write":
        kv = list(_kv_inputs(c, seed))
        st["k"], st["v"] = torch.stack([k for k, _ in kv]), torch.stack([v for _, v in kv])
    st.update(_other_inputs(c, seed))
    if c["op"] == "evict":
        w = st["kv4"].weights() if own else st["w"]
        w[:, :, :c["L"]] = st["w_in"]
    return st


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    return _run_write(state) if op == "write" else _run_evict(state) if op == "evict" \
        else _run_attend(state)


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    H, d, n, G = c["Hkv"], c["d"], c["n"], c["Hq"] // c["Hkv"]
    Ls = _lengths(c)
    row = 2 * (d // 2 + d // 8)          # K and V of one cached token and KV head
    tokens = sum(Ls)
    if c["op"] == "write":
        # x read, codes written, and the values written back
        return {"bytes": tokens * H * (2 * d * es + row) + c["B"] * c["L"] * H * 2 * d * es,
                "flops": tokens * H * 2 * d * 6}
    if c["op"] == "evict":
        kept = sum(min(L + n, c["budget"]) for L in Ls)
        gone = sum(max(0, L + n - c["budget"]) for L in Ls)
        # new rows read and written; every weight and position read; at most as many rows
        # moved as go; the kept values, positions and weights written out
        return {"bytes": H * (c["B"] * n * (2 * d * es + row) + (tokens + c["B"] * n) * 8
                              + min(gone, kept) * row) + H * c["B"] * c["budget"] * (2 * d * es)
                + H * kept * row,
                "flops": H * c["B"] * (n + c["budget"]) * 2 * d * 3}
    rows = c["B"] * n * c["Hq"] * d
    # a chunk's row sees the tokens up to itself
    pairs = sum(L * n - n * (n - 1) // 2 for L in Ls) * c["Hq"]
    acc = 2 * 4 * tokens * H if c["acc"] else 0
    return {"bytes": tokens * H * row + 2 * rows * es + acc, "flops": 4 * pairs * d}


# ---------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------
def _value64(x):
    """The value that the 4-bit cache holds for x [.., d], in 64 bits."""
    y = x.double().reshape(*x.shape[:-1], -1, GROUP)
    least, most = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    step = torch.exp2(torch.frexp(least)[1].double() - 8)      # bf16 spacing at `least`
    lo = torch.floor(least / step) * step
    s = (most - lo) / 15
    step = torch.exp2(torch.frexp(s)[1].double() - 8)
    s = torch.ceil(s / step) * step
    code = torch.where(s > 0, torch.round((y - lo) / s.clamp(min=1e-300)), 0.0)
    return (lo + s * code).reshape(x.shape)


def _exact_attend(c, seed):
    H, n, G, d = c["Hkv"], c["n"], c["Hq"] // c["Hkv"], c["d"]
    q = _other_inputs(c, seed)["q"]
    out = torch.zeros(c["B"], n, c["Hq"], d, dtype=torch.float64, device=DEV)
    w = torch.zeros(c["B"], H, c["L"], dtype=torch.float64, device=DEV)
    rows = (c["acc"] if c["op"] == "chunk" else 1) if c["acc"] else 0
    for b, (k, v) in enumerate(_kv_inputs(c, seed)):
        L = _lengths(c)[b]
        for h in range(H):
            K, V = _value64(k[h, :L]), _value64(v[h, :L])
            for g in range(G):
                s = q[b, :, h * G + g].double() @ K.T / math.sqrt(d)
                if n > 1:
                    s += torch.full((n, L), -math.inf, dtype=torch.float64,
                                    device=DEV).triu_(L - n + 1)
                p = torch.softmax(s, -1)
                out[b, :, h * G + g] = p @ V
                if rows:
                    w[b, h, :L] += p[n - rows:].sum(0)
    return {"out": out, "weights": w} if c["acc"] else {"out": out}


def _exact_evict(c, seed):
    x = _other_inputs(c, seed)
    B, H, keep = c["B"], c["Hkv"], c["budget"]
    k_out = torch.zeros(B, H, keep, c["d"], dtype=torch.float64, device=DEV)
    v_out, w_out = torch.zeros_like(k_out), torch.zeros(B, H, keep, dtype=torch.float64, device=DEV)
    p_out = torch.zeros(B, H, keep, dtype=torch.int32, device=DEV)
    Ls = _lengths(c)
    for b, (k, v) in enumerate(_kv_inputs(c, seed)):
        L, total = Ls[b], Ls[b] + c["n"]
        for h in range(H):
            K = torch.cat([_value64(k[h, :L]), _value64(x["k_new"][b, h])])
            V = torch.cat([_value64(v[h, :L]), _value64(x["v_new"][b, h])])
            w = x["w_in"][b, h, :L].tolist() + [0.0] * c["n"]
            rank = sorted(range(total), key=lambda t: (
                not (t < c["first"] or t >= total - c["recent"]), -w[t], t))
            rank = [t for t in rank if t < c["first"] or t >= total - c["recent"]] + \
                   [t for t in rank if not (t < c["first"] or t >= total - c["recent"])]
            stay = set(rank[:keep])
            where = list(range(min(total, keep)))
            late = iter(sorted(t for t in stay if t >= keep))
            where = [t if t in stay else next(late) for t in where]
            m = len(where)
            at = torch.tensor(where, device=DEV)
            k_out[b, h, :m], v_out[b, h, :m] = K[at], V[at]
            w_out[b, h, :m] = torch.tensor(w, dtype=torch.float64, device=DEV)[at]
            p_out[b, h, :m] = at.int()
    return {"k": k_out, "v": v_out, "positions": p_out, "weights": w_out,
            "lengths": torch.tensor([min(L + c["n"], keep) for L in Ls], device=DEV)}


def exact(case, seed):
    c = dict(case)
    if c["op"] == "evict":
        return _exact_evict(c, seed)
    if c["op"] != "write":
        return _exact_attend(c, seed)
    out = {"k": [], "v": []}
    for b, kv in enumerate(_kv_inputs(c, seed)):
        for name, x in zip(("k", "v"), kv):
            y = _value64(x)
            y[:, _lengths(c)[b]:] = 0
            out[name].append(y)
    return {name: torch.stack(x) for name, x in out.items()}
