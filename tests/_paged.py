"""A plain model of the paged cache for the tests: one CPU oracle cache per
sequence, the pages each kv head still holds, and attention, page weights and
eviction in 64 bits -- with the bounds that the kernels' roundings allow."""
import math

import numpy as np
import torch

import oracle
from bit_kv_cache_06_gb300 import kivi, paged

D = 128
HALF = 2.0 ** -11            # half a step of fp16, relative


class Model:
    def __init__(self, B, Hkv, g, bits=2, G=32, R=64, sink=0, meta=0, flush=0, fp8=0, columns=16,
                 max_new=64, seed=0, spare=5):
        self.B, self.Hkv, self.g, self.G, self.R, self.sink, self.flush = B, Hkv, g, G, R, sink, flush
        self.scales = (0.75, 0.5)
        cap = -(-columns * G // R) * R
        self.oc = [oracle.OracleCache(Hkv, D, bits, G, R, cap + 64 * R, Ns=sink, meta=meta, flush=flush,
                                      fp8=fp8, fp8_k_scale=0.75, fp8_v_scale=0.5) for _ in range(B)]
        self.columns = cap // G
        P = B * Hkv
        self.held = [[] for _ in range(P)]           # record numbers each pair still holds, in order
        shape = kivi.CacheShape(bits, G, R, B, g * Hkv, Hkv, D, cap, sink, meta, flush, fp8, 0.75, 0.5)
        self.num_pages = P * self.columns + spare
        gen = torch.Generator().manual_seed(seed)
        self.gen = gen
        table = torch.randperm(self.num_pages, generator=gen)[:P * self.columns].view(P, -1).int()
        rec = kivi.history_record_bytes(shape.params())
        rows = sink + R
        # unwritten memory is filled with NaN patterns: nothing may read it
        self.gpu = paged.KiviPagedCache(shape, self.num_pages, max_new=max_new, buffers=(
            torch.full((self.num_pages, rec), 0xff, dtype=torch.uint8, device="cuda"),
            torch.full((P, rows, D), float("nan"), dtype=torch.float16, device="cuda"),
            torch.full((P, rows, D), float("nan"), dtype=torch.float16, device="cuda"),
            table.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"),
            torch.zeros(B, dtype=torch.int32, device="cuda")))
        self.outlier = torch.where(torch.rand((Hkv, D), generator=gen) < 0.02, 30.0, 1.0)

    # ---- inputs: q, k, v as slices of one buffer, with rows behind the last sequence
    def chunk(self, counts, pad=3, scales=(1.0, 1.0, 1.0)):
        n, H = sum(counts), self.g * self.Hkv
        x = torch.randn((n + pad, H + 2 * self.Hkv, D), generator=self.gen)
        x[:, H:H + self.Hkv] *= self.outlier
        for i, (lo, hi) in enumerate(((0, H), (H, H + self.Hkv), (H + self.Hkv, H + 2 * self.Hkv))):
            x[:, lo:hi] *= scales[i]
        x[n:] = float("nan")                          # rows of no sequence
        qkv = x.half()
        self.counts = list(counts)
        off = np.concatenate([[0], np.cumsum(counts)])
        dev = qkv.cuda()
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + self.Hkv], qkv[:, H + self.Hkv:]
        self.dev = dict(q=dev[:, :H], k=dev[:, H:H + self.Hkv], v=dev[:, H + self.Hkv:],
                        offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_new=max(counts))
        self.off = off
        return self.dev

    def append(self):
        """The chunk enters the model (the GPU call is the test's)."""
        for b, oc in enumerate(self.oc):
            lo, hi = self.off[b], self.off[b + 1]
            if hi == lo:
                continue
            was = oc.n_quant
            assert oc.prefill(self.k[lo:hi].transpose(0, 1).contiguous().numpy(),
                              self.v[lo:hi].transpose(0, 1).contiguous().numpy()) == 0
            for h in range(self.Hkv):
                self.held[b * self.Hkv + h] += list(range(was // self.G, oc.n_quant // self.G))

    def check_state(self):
        """Pages, rows and counts equal the oracle's, byte for byte."""
        c = self.gpu
        table, pool = c.table.cpu().numpy(), c.pool.cpu().numpy()
        kr, vr = (x.cpu().numpy().view(np.uint16) for x in (c.k_fp16, c.v_fp16))
        tokens, gone = c.n_tokens.tolist(), c.n_evicted.tolist()
        for b, oc in enumerate(self.oc):
            assert tokens[b] == oc.n_tokens, (b, tokens[b], oc.n_tokens)
            head = oc.n_quant % self.R
            ring = [self.sink + (head + i) % self.R for i in range(oc.n_resid)]
            for h in range(self.Hkv):
                p = b * self.Hkv + h
                assert gone[b] == oc.n_quant // self.G - len(self.held[p])
                if self.held[p]:
                    ref = oc.export_history(h)[self.held[p]]
                    got = pool[table[p, :len(self.held[p])]]
                    assert np.array_equal(got, ref), f"pages of pair {p}"
                for got, s, r in ((kr, oc.kr, oc.kres), (vr, oc.vr, oc.vres)):
                    assert np.array_equal(got[p, :oc.n_sink], s[h, :oc.n_sink]), f"sink rows of pair {p}"
                    assert np.array_equal(got[p, ring], r[h, :oc.n_resid]), f"window of pair {p}"
            assert len(set(table[b * self.Hkv].tolist())) == self.columns
        assert c.status() == 0

    # ---- plain attention
    def keys(self, b, h, new=True):
        """K, V of everything the chunk's tokens may see (64 bits), how many
        of them are cached, and which are page tokens (first, count)."""
        oc, p = self.oc[b], b * self.Hkv + h
        ns, nr = oc.n_sink, oc.n_resid

        def f16(x):
            return torch.from_numpy(np.ascontiguousarray(x).view(np.float16).astype(np.float64))

        parts = []
        for sink, deq, res, fresh in ((oc.kr, oc.dequant_k, oc.kres, self.k), (oc.vr, oc.dequant_v, oc.vres, self.v)):
            deep = torch.from_numpy(np.asarray(deq(h))).double()[ns:ns + oc.n_quant]
            pages = deep.view(-1, self.G, D)[self.held[p]].reshape(-1, D)
            x = [f16(sink[h, :ns]), pages, f16(res[h, :nr])]
            if new:
                x.append(fresh[self.off[b]:self.off[b + 1], h].double())
            parts.append(torch.cat(x))
        n = self.counts[b] if new else 0
        return parts[0], parts[1], parts[0].shape[0] - n, (ns, len(self.held[p]) * self.G)

    def softmax(self, b, i, K, cached, cap, causal, tau=None):
        """Probabilities [T, n] of query head i, and a bound on every score's
        size sum |q k| tau."""
        q = self.q[self.off[b]:self.off[b + 1], i].double()
        tau = 1.0 / math.sqrt(D) if tau is None else tau
        s = q @ K.T * tau
        size = q.abs() @ K.abs().T * tau
        if cap > 0:
            s = cap * torch.tanh(s / cap)
        if causal:
            t = torch.arange(q.shape[0])[:, None]
            j = torch.arange(K.shape[0])[None] - cached
            s = s.masked_fill(j > t, -math.inf)
        m = s.amax(1, keepdim=True) if K.shape[0] else torch.zeros((q.shape[0], 1), dtype=torch.float64)
        e = torch.exp(s - m)
        return e / e.sum(1, keepdim=True).clamp_min(1e-300), size

    def attention(self, cap=0.0, causal=True, new=True, key_eps=HALF, tau=None):
        """Rows [N, Hq, D] and how far a kernel may be off each element.
        Roundings: dequantised keys to fp16 (key_eps), values to fp16, their
        scale first (2 HALF), the probabilities to fp16 (HALF), the output to
        fp16 (HALF); fp32 sums
        (2^-14 covers products and sums of a few thousand terms); the cap's
        tanh (cap 2^-21).  A score error d moves p_j by at most p_j (e^(2d) - 1).
        Below 2^-14 fp16 has a fixed step of 2^-24, half of which, 2^-25, is
        what a rounding is off there whatever the number's size: once for the
        output, twice for each value, which is carried halved (times its p,
        which sum to 1), and once for each 2^(s_j - m) it multiplies, the
        divisor being 1 or more: that adds 2^-25 (3 + sum_j |v_j|) over the
        tokens a row sees.
        Few query rows: o = sum p s code - sum p s z, two fp32 sums of up to 64
        slices each (64 steps of 2^-24) whose terms are at most 4 max_c |v_jc|
        in size (a group's codes span its range, at most twice its largest
        value; so do z s): 2^-18 sum_j p_j 4 max_c |v_jc|."""
        out = torch.zeros((self.off[-1], self.g * self.Hkv, D), dtype=torch.float64)
        tol = torch.zeros_like(out)
        for b in range(self.B):
            if self.counts[b] == 0:
                continue
            for h in range(self.Hkv):
                K, V, cached, _ = self.keys(b, h, new)
                for i in range(h * self.g, (h + 1) * self.g):
                    p, size = self.softmax(b, i, K, cached, cap, causal, tau)
                    o = p @ V
                    d = (key_eps + 2.0 ** -18) * size + cap * 2.0 ** -21
                    dp = p * torch.expm1(2 * torch.where(p > 0, d, torch.zeros_like(d)))
                    sl = slice(self.off[b], self.off[b + 1])
                    out[sl, i] = o
                    seen = (p > 0).double()
                    tol[sl, i] = (2.0 ** -16 * (p @ V.abs().amax(1, keepdim=True)) + 2.0 ** -25 * (3 + seen @ V.abs()) + HALF * o.abs() + (3 * HALF + 2.0 ** -14) * (p @ V.abs()) + dp @ V.abs() +
                                  dp.sum(1, keepdim=True) * o.abs())
        return out, tol

    def weights(self, cap=0.0, causal=True, new=True, base=None):
        """Page weights [P, C] added to base, and the bound: keys carried with
        22 bits and fp32 sums (2^-19 of a score's size), log2 and 2^x of
        numbers up to 2^7 in fp32 (2^-16), the sums themselves (2^-18)."""
        P = self.B * self.Hkv
        w = torch.zeros((P, self.columns), dtype=torch.float64) if base is None else base.double().clone()
        tol = w.abs() * 2.0 ** -22 + 1e-30
        for b in range(self.B):
            if self.counts[b] == 0:
                continue
            for h in range(self.Hkv):
                K, V, cached, (first, n) = self.keys(b, h, new)
                for i in range(h * self.g, (h + 1) * self.g):
                    p, size = self.softmax(b, i, K, cached, cap, causal)
                    if n == 0:
                        continue
                    d = torch.where(p > 0, 2.0 ** -19 * size, torch.zeros_like(size)).amax(1, keepdim=True) + cap * 2.0 ** -21
                    rel = 2 * d + 2.0 ** -16 + 2.0 ** -18
                    part = p[:, first:first + n].view(p.shape[0], -1, self.G).sum(2)
                    w[b * self.Hkv + h, :n // self.G] += part.sum(0)
                    tol[b * self.Hkv + h, :n // self.G] += (part * rel).sum(0) + 2.0 ** -24
        return w, tol

    def evict(self, table, weights, budget, recent):
        """Plain eviction of numpy table and weights [P, C]; updates `held`."""
        table, weights = table.copy(), weights.copy()
        for p in range(self.B * self.Hkv):
            n = len(self.held[p])
            if n <= budget:
                continue
            keep, drop = pick(weights[p][:n], budget, recent)
            table[p, :n] = [table[p, i] for i in keep + drop]
            weights[p, :n] = [weights[p, i] for i in keep] + [0.0] * len(drop)
            self.held[p] = [self.held[p][i] for i in keep]
        return table, weights


def pick(w, budget, recent):
    n, recent = len(w), min(recent, budget)
    key = [(-math.inf if math.isnan(x) else x) for x in w]
    order = sorted(range(n - recent), key=lambda i: (math.isnan(w[i]), -key[i], i))
    best = sorted(order[:budget - recent])
    keep = best + list(range(n - recent, n))
    return keep, sorted(set(range(n)) - set(keep))
