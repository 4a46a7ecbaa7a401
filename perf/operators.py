"""Cases of the paged-cache operators, in their plain form and through the library.

A paged cache keeps a quantised KV cache in pages of one key-group record each
(include/kivi.h, "history": G tokens of one kv head), a table row of page
numbers for every (sequence, kv head), and the newest and first tokens in fp16
rows.  Four operators work on it:

  attention  new tokens of a ragged batch attend to their sequence's cached
             tokens and, causally, to one another
  weights    the softmax weights of such an attention, summed per page
  evict      the pages with the least accumulated weight leave a sequence
  append     new tokens enter the cache; whole key groups are quantised

The plain forms work on dense, padded tensors with validity masks.
"""
import math

import torch

own = False

D = 128
KINDS = {"2bit": (2, 0), "4bit": (4, 0), "e4m3": (8, 1), "e5m2": (8, 2)}


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # the smallest call: one sequence of one kv head, a short context (latency)
        dict(name="attend tiny", op="attention", B=1, Hq=4, Hkv=1, kind="2bit", G=32, R=32, sink=0,
             meta=0, ctx=288, ragged=0, T=1, softcap=0.0),
        # serving: one new token for each of eight sequences of up to 32k tokens
        dict(name="attend decode", op="attention", B=8, Hq=32, Hkv=8, kind="2bit", G=32, R=128, sink=0,
             meta=0, ctx=32768, ragged=1, T=1, softcap=0.0),
        # verifying drafted tokens: up to eight new tokens for many sequences, capped scores
        dict(name="attend verify", op="attention", B=32, Hq=32, Hkv=8, kind="4bit", G=64, R=128, sink=4,
             meta=0, ctx=8192, ragged=1, T=8, softcap=30.0),
        # a scheduler's mixed step over FP8 pages: ragged chunks, eight query heads to a kv head
        dict(name="attend mixed fp8", op="attention", B=4, Hq=64, Hkv=8, kind="e4m3", G=32, R=128, sink=0,
             meta=0, ctx=16384, ragged=1, T=512, softcap=0.0),
        # a chunk of a long prompt: 2048 new tokens after 32k cached ones
        dict(name="attend chunk", op="attention", B=1, Hq=32, Hkv=8, kind="2bit", G=32, R=128, sink=0,
             meta=1, ctx=32768, ragged=0, T=2048, softcap=0.0),
        # every decode step adds its weights to the pages' totals
        dict(name="weigh decode", op="weights", B=8, Hq=32, Hkv=8, kind="2bit", G=32, R=128, sink=0,
             meta=0, ctx=32768, ragged=1, T=1, softcap=0.0),
        # the last 32 tokens of two prompts vote on what to keep
        dict(name="weigh window", op="weights", B=2, Hq=32, Hkv=8, kind="4bit", G=64, R=128, sink=4,
             meta=1, ctx=16384, ragged=1, T=32, softcap=30.0),
        # eight sequences are cut to half their pages
        dict(name="evict half", op="evict", B=8, Hkv=8, cols=1024, held=1020, ragged=1, budget=512, recent=32),
        # a million tokens are cut to a quarter
        dict(name="evict long", op="evict", B=1, Hkv=8, cols=32768, held=32764, ragged=0, budget=8192,
             recent=64),
        # prompts of up to 8k tokens enter an empty cache
        dict(name="append prompts", op="append", B=8, Hkv=8, kind="2bit", G=32, R=128, sink=4, meta=0,
             ctx=0, ragged=1, T=8192),
        # short prompts, 4-bit pages with fp16 scales
        dict(name="append short", op="append", B=3, Hkv=4, kind="4bit", G=64, R=64, sink=0, meta=1,
             ctx=0, ragged=1, T=333),
        # one decoded token for each of 32 sequences (no window is full)
        dict(name="append tokens", op="append", B=32, Hkv=8, kind="4bit", G=64, R=128, sink=0, meta=0,
             ctx=2000, ragged=0, T=1),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "weights", "evict", "append"])
    if op == "evict":
        B, Hkv = _logint(rng, 1, 16), rng.choice([1, 2, 4, 8])
        held = _logint(rng, 8, 262144 // (B * Hkv))
        budget = rng.randint(1, held)
        return dict(op=op, B=B, Hkv=Hkv, cols=held + rng.randint(0, 9), held=held, ragged=rng.randint(0, 1),
                    budget=budget, recent=rng.randint(0, min(budget, 64)))
    kind = rng.choice(["2bit", "2bit", "4bit", "4bit", "e4m3", "e5m2"])
    G = 32 if kind[0] == "e" else rng.choice([16, 32, 64, 128])
    c = dict(op=op, kind=kind, G=G, R=G * rng.choice([1, 2, 4]) if G < 128 else 128,
             sink=rng.choice([0, 0, 4, 37]), meta=0 if kind[0] == "e" else rng.choice([0, 1]),
             ragged=rng.randint(0, 1), Hkv=rng.choice([1, 2, 4, 8]))
    if op == "append":
        T = _logint(rng, 1, 8192)
        return dict(c, B=_logint(rng, 1, max(1, min(32, 65536 // T))), ctx=0, T=T)
    g = rng.choice([1, 2, 4, 5, 8])
    T = _logint(rng, 1, 64 if op == "weights" else 1024)
    ctx = _logint(rng, 1, 32768) if rng.random() < 0.9 else 0
    most = min(32, (1 << 27) // ((ctx + T) * D * c["Hkv"]), (1 << 30) // ((ctx + T) * T * c["Hkv"] * g))
    return dict(c, B=_logint(rng, 1, max(1, most)), Hq=g * c["Hkv"], ctx=ctx, T=T,
                softcap=rng.choice([0.0, 0.0, 20.0, 50.0]))


# ------------------------------------------------------------------ layout ---

def _lengths(c):
    """Cached and new tokens of each sequence, from the case alone."""
    B = c["B"]
    if not c["ragged"]:
        return [c["ctx"]] * B, [c["T"]] * B
    # sequence 0 is the longest; the others spread over the upper half
    ctx = [c["ctx"] - (c["ctx"] // 2) * ((7 * b) % B) // B for b in range(B)]
    new = [c["T"] - (c["T"] // 2) * ((5 * b) % B) // B for b in range(B)]
    return ctx, new


def _split(n, c):
    """Sink tokens, quantised tokens and window tokens of n tokens (whole-window flush)."""
    s = min(n, c["sink"])
    m = n - s
    q = (m - 1) // c["R"] * c["R"] if m > 0 else 0
    return s, q, m - q


def _columns(c):
    ctx, new = _lengths(c)
    most = max(a + b for a, b in zip(ctx, new))
    return -(-most // c["R"]) * c["R"] // c["G"]


class Layout:
    """Byte positions inside a record (include/kivi.h)."""

    def __init__(self, c):
        self.bits, self.fmt = KINDS[c["kind"]]
        self.G, self.meta = c["G"], c["meta"]
        if self.fmt:
            self.bytes = 64 * D
            return
        self.SL, self.RB, self.VG = min(self.G, 32), D * self.bits // 8, D // self.G
        self.w = 2 if self.meta else 4
        self.head = 2 * self.w * D
        self.sub = self.SL * (2 * self.RB + 2 * self.w * self.VG)
        self.bytes = self.head + self.G // self.SL * self.sub
        ch = torch.arange(D)
        run = self.G // 8
        if run * self.bits < 8:
            self.pos = ch
        else:
            u = ch % self.G
            self.pos = 16 * (u // run) + run * (ch // self.G) + u % run

    @property
    def ftype(self):
        return torch.float16 if self.meta else torch.float32


_FP8 = {1: (torch.float8_e4m3fn, 448.0), 2: (torch.float8_e5m2, 57344.0)}
K8, V8 = 0.75, 0.625        # FP8 scales of the cases


def _over(x, n):
    """x / n, rounded once (a division by a Python number would multiply by its reciprocal)."""
    return x / torch.full_like(x, n)


def _quant(x, axis, lay):
    """Scale, zero point and codes of x (fp32), grouped along `axis`."""
    lo, hi = x.amin(axis, keepdim=True), x.amax(axis, keepdim=True)
    top = float(2 ** lay.bits - 1)
    s = _over(hi - lo, top)
    if lay.meta:
        s = torch.maximum(s, lo.abs() * 2.0 ** -11).clamp_min(2.0 ** -24)
        h = s.half()
        up = torch.where(h.float() < s, (h.view(torch.int16) + 1).view(torch.float16), h)
        s = up.float()
    else:
        s = s.clamp_min(1e-8)
    z = torch.round(-lo / s) + 0.0
    return s, z, (torch.round(x / s) + z).clamp_(0, top).to(torch.uint8)


def _pack(codes, bits):
    per = 8 // bits
    v = codes.unflatten(-1, (-1, per))
    out = v[..., 0].clone()
    for i in range(1, per):
        out |= v[..., i] << (bits * i)
    return out


def _records(k, v, lay):
    """Records [..., n, bytes] of whole key groups k, v: fp16 [..., n, G, D]."""
    if lay.fmt:
        t, top = _FP8[lay.fmt]
        two = [_over(x.float(), s).clamp_(-top, top).to(t).view(torch.uint8).flatten(-2) for x, s in ((k, K8), (v, V8))]
        return torch.cat(two, -1)
    ks, kz, kc = _quant(k.float(), -2, lay)
    vs, vz, vc = (x.flatten(-2) for x in _quant(v.float().unflatten(-1, (lay.VG, lay.G)), -1, lay))
    order = torch.empty_like(lay.pos)
    order[lay.pos] = torch.arange(D)
    kc, vc = _pack(kc, lay.bits), _pack(vc[..., order.to(vc.device)], lay.bits)

    def raw(x):
        return x.to(lay.ftype).contiguous().view(torch.uint8)

    def subs(x):                                    # [..., n, G, w] -> [..., n, G / SL, SL * w]
        return x.unflatten(-2, (-1, lay.SL)).flatten(-2)

    sub = torch.cat([subs(kc), subs(vc), subs(raw(vs)), subs(raw(vz))], -1)
    return torch.cat([raw(ks.squeeze(-2)), raw(kz.squeeze(-2)), sub.flatten(-2)], -1)


# ------------------------------------------------------------------ inputs ---

def _rand(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda")


def _kv(shape, kmul, gen):
    """Keys with a few channels far larger than the rest, values with a few such tokens."""
    k = (_rand(shape, gen) * kmul).half()
    v = _rand(shape, gen)
    v *= torch.where(torch.rand(shape[:-1] + (1,), generator=gen, device="cuda") < 0.005, 200.0, 1.0)
    return k, v.half()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    if c["op"] == "evict":
        return _prepare_evict(c, gen)
    lay, B, Hkv = Layout(c), c["B"], c["Hkv"]
    P, cols, rows = B * Hkv, _columns(c), c["sink"] + c["R"]
    ctx, new = _lengths(c)
    held = [_split(n, c)[1] // c["G"] for n in ctx]
    chans = torch.rand((Hkv, D), generator=gen, device="cuda").argsort(-1) < 3
    kmul = torch.where(chans, 50.0, 1.0)[:, None]                      # [Hkv, 1, D]

    # the pool holds more pages than the rows name, in no order
    num_pages = P * cols + 7
    pool = torch.zeros((num_pages, lay.bytes), dtype=torch.uint8, device="cuda")
    table = torch.randperm(num_pages, generator=gen, device="cuda")[:P * cols].view(P, cols).int()
    k_rows = torch.zeros((P, rows, D), dtype=torch.float16, device="cuda")
    v_rows = torch.zeros_like(k_rows)
    for b in range(B):
        s, q, r = _split(ctx[b], c)
        k, v = _kv((Hkv, ctx[b], D), kmul, gen)
        at = slice(b * Hkv, (b + 1) * Hkv)
        if held[b]:
            rec = _records(k[:, s:s + q].unflatten(1, (-1, c["G"])), v[:, s:s + q].unflatten(1, (-1, c["G"])), lay)
            pool[table[at, :held[b]].long().flatten()] = rec.flatten(0, 1)
        for buf, x in ((k_rows, k), (v_rows, v)):
            buf[at, :s] = x[:, :s]
            buf[at, c["sink"]:c["sink"] + r] = x[:, s + q:]
    N = sum(new)
    x = _rand((N, c.get("Hq", 0) + 2 * Hkv, D), gen)                   # one projection's output: q, k, v side by side
    Hq = c.get("Hq", 0)
    x[:, Hq:Hq + Hkv] *= kmul.transpose(0, 1)
    qkv = x.half()
    st = dict(case=c, lay=lay, pool=pool, k_rows=k_rows, v_rows=v_rows, table=table,
              n_tokens=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
              n_evicted=torch.zeros(B, dtype=torch.int32, device="cuda"),
              q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:],
              offsets=torch.tensor([0] + [sum(new[:b + 1]) for b in range(B)], dtype=torch.int32, device="cuda"),
              max_new=max(new), max_cached=max(ctx), new=new, ctx=ctx)
    st["n_start"] = st["n_tokens"].clone()
    if c["op"] == "weights":
        st["weights"] = torch.rand((P, cols), generator=gen, device="cuda")
    if own:
        from bit_kv_cache_06_gb300 import kivi, paged
        shape = kivi.CacheShape(lay.bits, c["G"], c["R"], B, Hq or Hkv, Hkv, D, cols * c["G"], c["sink"], c["meta"],
                                kivi.KIVI_FLUSH_WINDOW, lay.fmt, K8, V8)
        st["cache"] = paged.KiviPagedCache(shape, num_pages, max_new=max(new),
                                           buffers=(pool, k_rows, v_rows, table, st["n_tokens"], st["n_evicted"]))
    return st


def _held(c):
    """Pages that each sequence of an eviction holds."""
    return [c["held"] - c["ragged"] * ((5 * b) % 8) * c["held"] // 16 for b in range(c["B"])]


def _prepare_evict(c, gen):
    B, P, cols = c["B"], c["B"] * c["Hkv"], c["cols"]
    held = _held(c)
    # heavy-tailed weights, a few of them equal
    w = torch.rand((P, cols), generator=gen, device="cuda").pow(8.0)
    w[:, 1::17] = 0.25
    start = torch.randperm(P * cols, generator=gen, device="cuda").int()
    start = torch.cat([start, torch.zeros(B, dtype=torch.int32, device="cuda"), w.flatten().view(torch.int32)])
    # a window of 32 tokens follows the quantised ones, so held * 32 + 1 tokens have `held` pages
    tokens = torch.tensor([h * 32 + 1 for h in held], dtype=torch.int32, device="cuda")
    work = torch.empty_like(start)
    st = dict(case=c, start=start, work=work, table=work[:P * cols].view(P, cols),
              n_evicted=work[P * cols:P * cols + B], weights=work[P * cols + B:].view(torch.float32).view(P, cols),
              held=torch.tensor(held, device="cuda"), n_tokens=tokens)
    if own:
        from bit_kv_cache_06_gb300 import kivi, paged
        shape = kivi.CacheShape(2, 32, 32, B, c["Hkv"], c["Hkv"], D, cols * 32)
        pool = torch.empty((P * cols, 4096), dtype=torch.uint8, device="cuda")
        rows = torch.empty((P, 32, D), dtype=torch.float16, device="cuda")
        st["cache"] = paged.KiviPagedCache(shape, P * cols, max_new=1,
                                           buffers=(pool, rows, rows.clone(), st["table"], tokens, st["n_evicted"]))
    return st


# --------------------------------------------------------------------- run ---

def run(state):
    op = state["case"]["op"]
    if op == "attention":
        return _attend(state)
    if op == "weights":
        return _weigh(state)
    if op == "evict":
        return _evict(state)
    return _append(state)


def _attend(st):
    c = st["case"]
    if own:
        return st["cache"].attention(st["q"], st["k"], st["v"], st["offsets"], max_new=st["max_new"],
                                     max_cached=st["max_cached"], softcap=c["softcap"])
    q, keys, valid = _keys(st)
    p = _probs(q, keys, valid, c["softcap"])
    vals = torch.cat([st["v_rows"].unflatten(0, (c["B"], -1)).float(), _pages(st, 1), _padded(st, "v")], 2)
    o = (p.flatten(3, 4).transpose(2, 3) @ vals).unflatten(2, (-1, st["max_new"]))   # [B, Hkv, g, T, D]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                                        # [B, T, Hq, D]
    return o[_where(st)].half()


def _weigh(st):
    c = st["case"]
    if own:
        w = st["weights"].clone()
        st["cache"].weights(w, st["q"], st["k"], st["offsets"], max_new=st["max_new"], max_cached=st["max_cached"],
                            softcap=c["softcap"])
        return w
    q, keys, valid = _keys(st)
    p = _probs(q, keys, valid, c["softcap"])                                          # [B, Hkv, keys, g, T]
    rows, cols = st["k_rows"].shape[1], st["table"].shape[1]
    live = _live(st)[:, None, None, None, :]
    mass = (p[:, :, rows:rows + cols * c["G"]] * live).sum((3, 4)).unflatten(2, (cols, -1)).sum(3)
    return st["weights"] + mass.flatten(0, 1)


def _evict(st):
    c = st["case"]
    st["work"].copy_(st["start"])
    table, weights, n_evicted = st["table"], st["weights"], st["n_evicted"]
    if own:
        st["cache"].evict(weights, c["budget"], c["recent"])
        return {"table": table, "n_evicted": n_evicted, "weights": weights}
    col = torch.arange(c["cols"], device="cuda")
    n = st["held"].repeat_interleave(c["Hkv"])[:, None]
    inside = col < n
    score = torch.where(col >= n - min(c["recent"], c["budget"]), math.inf, weights)
    score = torch.where(inside, score, -math.inf)
    rank = score.sort(dim=1, descending=True, stable=True).indices.argsort(1)
    kept = (rank < c["budget"]) & inside
    place = torch.where(n <= c["budget"], col, (~kept).int() + (~inside).int()).sort(dim=1, stable=True).indices
    gone = (n > c["budget"]) & inside & (col >= c["budget"])
    return {"table": table.gather(1, place),
            "n_evicted": n_evicted + (st["held"] - c["budget"]).clamp_min(0).int(),
            "weights": weights.gather(1, place).masked_fill(gone, 0.0)}


def _append(st):
    c, lay = st["case"], st["lay"]
    st["n_tokens"].copy_(st["n_start"])
    if own:
        st["cache"].append(st["k"], st["v"], st["offsets"], max_new=st["max_new"])
        return {"pool": st["pool"], "k_rows": st["k_rows"], "v_rows": st["v_rows"], "n_tokens": st["n_tokens"]}
    B, Hkv, G, R, S = c["B"], c["Hkv"], c["G"], c["R"], c["sink"]
    k, v = _padded(st, "k").half(), _padded(st, "v").half()                           # [B, Hkv, T, D]
    n0 = st["n_tokens"].long()
    n1 = n0 + (st["offsets"][1:] - st["offsets"][:-1])
    # tokens by their index in the sequence: the fp16 rows' old ones, then the new ones
    m1 = (n1 - S).clamp_min(0)
    q1 = torch.where(m1 > 0, (m1 - 1) // R * R, 0)
    k_rows, v_rows = (x.unflatten(0, (B, Hkv)) for x in (st["k_rows"], st["v_rows"]))
    if c["ctx"] == 0:
        # from an empty cache every quantised token is a new one: token S + G j + u
        cols = st["table"].shape[1]
        last = max(k.shape[2] - 1, 0)
        idx = (S + torch.arange(cols * G, device="cuda")).clamp_max(last)
        rec = _records(k[:, :, idx].unflatten(2, (cols, G)), v[:, :, idx].unflatten(2, (cols, G)), lay)
        due = (torch.arange(cols, device="cuda") < (q1 // G)[:, None])[:, None].expand(B, Hkv, cols)
        st["pool"][st["table"].unflatten(0, (B, Hkv))[due].long()] = rec[due]
    row = torch.arange(S + R, device="cuda")
    token = torch.where(row < S, row, row + q1[:, None])                              # [B, rows]
    fresh = (token >= n0[:, None]) & (token < n1[:, None])
    src = (token - n0[:, None]).clamp(0, k.shape[2] - 1)[:, None, :, None].expand(B, Hkv, S + R, D)
    for rows, x in ((k_rows, k), (v_rows, v)):
        rows.copy_(torch.where(fresh[:, None, :, None], x.gather(2, src), rows))
    st["n_tokens"].copy_(n1)
    return {"pool": st["pool"], "k_rows": st["k_rows"], "v_rows": st["v_rows"], "n_tokens": st["n_tokens"]}


# ------------------------------------------------------------- plain parts ---

def _where(st):
    """(sequence, place in it) of every new token."""
    at = torch.arange(st["q"].shape[0], device="cuda")
    b = torch.searchsorted(st["offsets"][1:].contiguous(), at.int(), right=True)
    return b, at - st["offsets"][b].long()


def _live(st):
    """[B, T]: which places of the padded batch hold a new token."""
    return torch.arange(st["max_new"], device="cuda") < (st["offsets"][1:] - st["offsets"][:-1])[:, None]


def _padded(st, name):
    """New tokens [N, H, D] as fp32 [B, H, T, D], zero where a sequence has no more."""
    x = st[name]
    out = torch.zeros((st["case"]["B"], st["max_new"]) + x.shape[1:], device="cuda")
    out[_where(st)] = x.float()
    return out.transpose(1, 2)


def _pages(st, part):
    """Keys (0) or values (1) of the pages: fp32 [B, Hkv, columns * G, D]."""
    c, lay = st["case"], st["lay"]
    rec = st["pool"][st["table"].long()]                                              # [P, cols, bytes]
    if lay.fmt:
        x = rec.unflatten(2, (2, 32, D))[:, :, part].contiguous().view(_FP8[lay.fmt][0]).float() * (K8, V8)[part]
        return x.flatten(1, 2).unflatten(0, (c["B"], -1))
    sub = rec[:, :, lay.head:].unflatten(2, (-1, lay.sub))
    n = lay.SL * lay.RB
    codes = sub[..., part * n:(part + 1) * n].unflatten(3, (lay.SL, lay.RB))
    shift = torch.arange(0, 8, lay.bits, device="cuda", dtype=torch.uint8)
    codes = ((codes[..., None] >> shift) & (2 ** lay.bits - 1)).flatten(-2)           # [P, cols, G / SL, SL, D]

    def floats(x):
        return x.contiguous().view(lay.ftype).float()

    if part == 0:
        sz = floats(rec[:, :, :lay.head]).unflatten(2, (2, 1, 1, D))
        x = (codes.float() - sz[:, :, 1]) * sz[:, :, 0]
    else:
        codes = codes[..., lay.pos.to(codes.device)]
        sz = floats(sub[..., 2 * n:]).unflatten(3, (2, lay.SL, lay.VG, 1))
        x = ((codes.float().unflatten(4, (lay.VG, lay.G)) - sz[:, :, :, 1]) * sz[:, :, :, 0]).flatten(-2)
    return x.flatten(1, 3).unflatten(0, (c["B"], -1))


def _keys(st):
    """Queries [B, Hkv, g, T, D], keys [B, Hkv, n, D] (rows, pages, new tokens) and which of them each
    new token sees, [B, n, T]."""
    c = st["case"]
    B, R, S = c["B"], c["R"], c["sink"]
    q = _padded(st, "q").unflatten(1, (c["Hkv"], -1))
    keys = torch.cat([st["k_rows"].unflatten(0, (B, -1)).float(), _pages(st, 0), _padded(st, "k")], 2)
    n = st["n_tokens"].long()[:, None]
    m = (n - S).clamp_min(0)
    flushed = torch.where(m > 0, (m - 1) // R * R, 0)
    row = torch.arange(S + R, device="cuda")
    rows = torch.where(row < S, row < n, row - S < m - flushed)
    pages = torch.arange(st["table"].shape[1] * c["G"], device="cuda") < flushed - st["n_evicted"].long()[:, None] * c["G"]
    cached = torch.cat([rows, pages], 1)[:, :, None].expand(-1, -1, st["max_new"])
    t = torch.arange(st["max_new"], device="cuda")
    among = ((t[:, None] <= t) & _live(st)[:, :, None])
    return q, keys, torch.cat([cached, among], 1)


def _probs(q, keys, valid, softcap):
    """Softmax weights [B, Hkv, n, g, T] of every query over the keys it sees."""
    s = keys @ q.flatten(2, 3).transpose(2, 3) * (1.0 / math.sqrt(D))                  # [B, Hkv, n, g T]
    s = s.unflatten(3, q.shape[2:4])
    if softcap > 0.0:
        s = softcap * torch.tanh(s / softcap)
    s = s.masked_fill(~valid[:, None, :, None, :], -math.inf)
    e = torch.exp(s - s.amax(2, keepdim=True).clamp_min(-3e38))
    return e / e.sum(2, keepdim=True).clamp_min(1e-30)


# -------------------------------------------------------------------- work ---

def work(case):
    c = case
    if c["op"] == "evict":
        n = sum(_held(c)) * c["Hkv"]
        # the rows' page numbers and weights, read and written once
        return {"bytes": 16.0 * n, "flops": 0.0}
    lay = Layout(c)
    ctx, new = _lengths(c)
    Hkv, N = c["Hkv"], sum(new)
    if c["op"] == "append":
        end = [_split(a + b, c)[1] - _split(a, c)[1] for a, b in zip(ctx, new)]
        kept = [min(b, sum(_split(a + b, c)[0::2])) for a, b in zip(ctx, new)]
        return {"bytes": float(Hkv * (N * 4 * D + sum(end) // c["G"] * lay.bytes + sum(kept) * 4 * D)), "flops": 0.0}
    parts = [_split(n, c) for n in ctx]
    pages, rows = sum(p[1] for p in parts) // c["G"], sum(p[0] + p[2] for p in parts)
    pairs = sum(a * b + b * (b + 1) // 2 for a, b in zip(ctx, new)) * c["Hq"]
    if c["op"] == "weights":
        # the records' key halves, the fp16 rows' keys, queries, new keys, and the pages' totals twice
        keys = lay.bytes // 2 if lay.fmt else lay.head + c["G"] * lay.RB
        return {"bytes": float(Hkv * (pages * keys + rows * 2 * D + N * 2 * D + pages * 8) + N * c["Hq"] * 2 * D),
                "flops": 2.0 * D * pairs}
    return {"bytes": float(Hkv * (pages * lay.bytes + rows * 4 * D + N * 4 * D) + N * c["Hq"] * 4 * D),
            "flops": 4.0 * D * pairs}


# ------------------------------------------------------------------- exact ---

def _exact_pages(st, pair, n, part):
    """Keys or values of the first n pages of a pair, element by element from the record's definition, fp64 [n G, D]."""
    lay, dev = st["lay"], "cuda"
    rec = st["pool"][st["table"][pair, :n].long()]
    if lay.fmt:
        at = part * 32 * D + torch.arange(32 * D, device=dev)
        return (rec[:, at].view(_FP8[lay.fmt][0]).double() * (K8, V8)[part]).reshape(-1, D)
    t = torch.arange(lay.G, device=dev)[:, None]
    ch = torch.arange(D, device=dev)[None]
    place = lay.pos.to(dev)[None] if part else ch
    base = lay.head + t // lay.SL * lay.sub
    byte = base + part * lay.SL * lay.RB + t % lay.SL * lay.RB + place * lay.bits // 8
    code = (rec[:, byte].int() >> (place * lay.bits % 8).int()) & (2 ** lay.bits - 1)

    def number(first, count):                       # number `count` of the array that begins at byte `first`
        at = (first + count * lay.w)[..., None] + torch.arange(lay.w, device=dev)
        return rec[:, at].contiguous().view(lay.ftype)[..., 0].double()

    if part == 0:
        zero = torch.zeros_like(ch)
        s, z = number(zero, ch), number(zero + lay.w * D, ch)
    else:
        first = base + 2 * lay.SL * lay.RB
        s = number(first + 0 * ch, t % lay.SL * lay.VG + ch // lay.G)
        z = number(first + lay.SL * lay.VG * lay.w + 0 * ch, t % lay.SL * lay.VG + ch // lay.G)
    return ((code.double() - z) * s).reshape(-1, D)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "evict":
        return _exact_evict(st)
    ctx, new, Hkv = st["ctx"], st["new"], c["Hkv"]
    if c["op"] == "append":
        # what the windows and sinks hold; the records are bytes
        out = [st["k_rows"].double(), st["v_rows"].double()]
        for b, at in enumerate(st["offsets"].tolist()[:-1]):
            s, q, r = _split(ctx[b] + new[b], c)
            for i in range(new[b]):
                n = ctx[b] + i
                row = n if n < c["sink"] else c["sink"] + n - s - q
                if row >= c["sink"] or n < c["sink"]:
                    for x, name in zip(out, ("k", "v")):
                        x[b * Hkv:(b + 1) * Hkv, row] = st[name][at + i].double()
        return {"pool": None, "k_rows": out[0], "v_rows": out[1], "n_tokens": torch.tensor([a + b for a, b in zip(ctx, new)])}
    g, first = c["Hq"] // Hkv, st["offsets"].tolist()
    out = torch.zeros((sum(new), c["Hq"], D), dtype=torch.float64, device="cuda")
    mass = st["weights"].double() if c["op"] == "weights" else None
    for b in range(c["B"]):
        s, nq, r = _split(ctx[b], c)
        t = torch.arange(new[b], device="cuda")
        for h in range(Hkv):
            pair, sl = b * Hkv + h, slice(first[b], first[b + 1])
            live = torch.cat([torch.arange(s, device="cuda"), c["sink"] + torch.arange(r, device="cuda")])
            parts = [[rows[pair, live].double(), _exact_pages(st, pair, nq // c["G"], i), x[sl, h].double()]
                     for i, (rows, x) in enumerate(((st["k_rows"], st["k"]), (st["v_rows"], st["v"])))]
            keys, vals = (torch.cat(x) for x in parts)
            for i in range(h * g, (h + 1) * g):
                z = st["q"][sl, i].double() @ keys.T / math.sqrt(D)
                if c["softcap"] > 0.0:
                    z = c["softcap"] * torch.tanh(z / c["softcap"])
                z[:, ctx[b]:].masked_fill_(t[None] > t[:, None], -math.inf)
                p = torch.softmax(z, 1)
                if mass is None:
                    out[sl, i] = p @ vals
                elif nq:
                    mass[pair, :nq // c["G"]] += p[:, s + r:s + r + nq].sum(0).view(-1, c["G"]).sum(1)
    return out if mass is None else mass


def _exact_evict(st):
    c = st["case"]
    P, cols = c["B"] * c["Hkv"], c["cols"]
    start = st["start"].cpu()
    table = start[:P * cols].view(P, cols).tolist()
    weights = start[P * cols + c["B"]:].view(torch.float32).view(P, cols).double().tolist()
    gone = [max(0, h - c["budget"]) for h in _held(c)]
    for p in range(P):
        n = _held(c)[p // c["Hkv"]]
        if n <= c["budget"]:
            continue
        recent = min(c["recent"], c["budget"])
        best = sorted(range(n - recent), key=lambda i: (-weights[p][i], i))[:c["budget"] - recent]
        keep = sorted(best) + list(range(n - recent, n))
        drop = sorted(set(range(n)) - set(keep))
        table[p][:n] = [table[p][i] for i in keep + drop]
        weights[p][:n] = [weights[p][i] for i in keep] + [0.0] * len(drop)
    return {"table": torch.tensor(table), "n_evicted": torch.tensor(gone), "weights": torch.tensor(weights, dtype=torch.float64)}
