"""Paged cache on the GPU against the plain model of tests/_paged.py: append,
attention of new tokens, page weights, eviction, and runs of them together."""
import ctypes
import math

import numpy as np
import pytest
import torch

from _paged import HALF, Model, pick
from bit_kv_cache_06_gb300 import kivi, paged, synth

pytestmark = pytest.mark.gpu

FORMATS = {
    "2bit-g32": dict(bits=2, G=32, R=64), "2bit-g16": dict(bits=2, G=16, R=32, sink=4),
    "2bit-g64-fp16meta": dict(bits=2, G=64, R=64, meta=1), "2bit-g128": dict(bits=2, G=128, R=128, columns=6),
    "4bit-g16-fp16meta": dict(bits=4, G=16, R=16, meta=1), "4bit-g32": dict(bits=4, G=32, R=128, flush=1),
    "4bit-g64": dict(bits=4, G=64, R=64, sink=37), "4bit-g128-fp16meta": dict(bits=4, G=128, R=128, meta=1, columns=6),
    "e4m3": dict(bits=8, G=32, R=32, fp8=1), "e5m2": dict(bits=8, G=32, R=96, fp8=2, flush=1, sink=5),
}


def close(got, want, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() > tol
    if bad.any():
        i = ((got - want).abs() / tol.clamp_min(1e-300)).argmax()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(got.flatten()[i])} for "
                             f"{float(want.flatten()[i])} +- {float(tol.flatten()[i]):.3g}")


def fill(m, *steps):
    """Append chunks of the given counts to the model and the cache."""
    for counts in steps:
        x = m.chunk(counts)
        m.gpu.append(x["k"], x["v"], x["offsets"], x["max_new"])
        m.append()


def attend(m, cap=0.0, causal=True, new=True, **kw):
    x = m.dev
    out = torch.full((x["q"].shape[0],) + tuple(x["q"].shape[1:]), 7.0, dtype=torch.float16, device="cuda")
    m.gpu.attention(x["q"], x["k"] if new else None, x["v"] if new else None, x["offsets"], x["max_new"],
                    softcap=cap, causal=causal, out=out, **kw)
    want, tol = m.attention(cap, causal, new)
    n = int(m.off[-1])
    assert (out[n:] == 7.0).all(), "rows of no sequence were written"
    close(out[:n], want, tol, "attention")
    return out


@pytest.mark.parametrize("name", FORMATS)
def test_append_writes_the_oracles_records(name):
    """Ragged chunks -- empty, one token, across a window's edge, several
    windows at once -- leave the records, rows and counts of the oracle."""
    kw = FORMATS[name]
    R = kw["R"]
    m = Model(4, 2, 1, seed=1, **kw)
    fill(m, [0, 1, R, R + 1])
    m.check_state()
    fill(m, [R + 3, 0, 1, 2 * R - 1], [1, 1, 1, 1], [2 * R, 3, R - 1, 0])
    m.check_state()
    for _ in range(3):
        fill(m, [1, 1, 1, 1])
    m.check_state()


@pytest.mark.parametrize("name", FORMATS)
def test_attention_and_weights_of_every_format(name):
    """A ragged chunk (8, 0, 1 and 70 new tokens) over empty, short and long
    sequences; pages end inside tiles."""
    kw = FORMATS[name]
    R = kw["R"]
    m = Model(4, 2, 4, seed=2, max_new=70, **kw)
    fill(m, [3 * R + 5, R, 0, 4 * R + 1])
    m.chunk([8, 0, 1, 70])
    attend(m)
    base = torch.rand((8, m.columns))
    w = base.cuda()
    x = m.dev
    m.gpu.weights(w, x["q"], x["k"], x["offsets"], x["max_new"])
    close(w, *m.weights(base=base), "weights")
    assert m.gpu.status() == 0


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 7, 8])
def test_query_groups(g):
    m = Model(2, 2, g, seed=3, max_new=33, sink=3)
    fill(m, [200, 77])
    m.chunk([33, 1])
    attend(m)
    m.chunk([1, 1])
    attend(m)
    x = m.dev
    w = torch.zeros((4, m.columns), device="cuda")
    m.gpu.weights(w, x["q"], x["k"], x["offsets"], x["max_new"])
    close(w, *m.weights(), "weights")


@pytest.mark.parametrize("cap", [0.0, 2.0, 30.0])
@pytest.mark.parametrize("causal,new", [(True, True), (False, True), (True, False)])
def test_caps_and_masks(cap, causal, new):
    m = Model(3, 2, 4, seed=4, max_new=90, bits=4, G=64, R=64)
    fill(m, [0, 65, 400])
    m.chunk([90, 17, 2])
    out = attend(m, cap, causal, new)
    if not new:
        assert (out[:90] == 0).all()              # an empty sequence: nothing to see
    base = torch.rand((6, m.columns))
    w, x = base.cuda(), m.dev
    m.gpu.weights(w, x["q"], x["k"] if new else None, x["offsets"], x["max_new"], softcap=cap, causal=causal)
    close(w, *m.weights(cap, causal, new, base), "weights")


@pytest.mark.parametrize("counts", [[1], [2], [15], [16], [17], [31], [63], [64], [65], [127], [128], [129],
                                    [255], [256], [257], [513]])
def test_chunk_lengths(counts):
    """Row tiles that are full, one short and one over, for first chunks too."""
    for g in (1, 4):
        m = Model(1, 1, g, seed=5, max_new=counts[0], columns=24)
        m.chunk(counts)
        attend(m)
        fill(m, [333])
        m.chunk(counts)
        attend(m)
        attend(m, softmax_scale=0.0, max_cached=333)   # a tight bound, another split


def test_long_cache_and_bounds():
    """20000 cached tokens: many splits, and any bound that holds."""
    m = Model(1, 1, 4, seed=6, columns=640, max_new=300, R=128)
    for _ in range(20):
        fill(m, [1000])
    for counts in ([1], [4], [40], [300]):
        m.chunk(counts)
        want, tol = m.attention()
        for hint in (0, 20000, 20001):
            x = m.dev
            close(m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], x["max_new"], max_cached=hint)[:counts[0]],
                  want, tol, f"{counts} {hint}")
        ref, wt = m.weights()
        for hint in (0, 20000, 20001):
            w = torch.zeros((1, m.columns), device="cuda")
            m.gpu.weights(w, x["q"], x["k"], x["offsets"], x["max_new"], max_cached=hint)
            close(w, ref, wt, f"weights {counts} {hint}")


def test_scale_is_the_callers():
    m = Model(1, 2, 2, seed=7)
    fill(m, [100])
    m.chunk([5])
    x = m.dev
    out = m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], 5, softmax_scale=0.5)
    close(out[:5], *m.attention(tau=0.5), "scale")


def test_new_form_of_the_decode():
    """A paged view of a KiviCache attends like kivi_decode_attention: both
    within the bound of the plain result, for every storage."""
    for kw in (dict(bits=2, G=32, R=128), dict(bits=4, G=64, R=64, meta=1), dict(bits=8, G=32, R=64, fp8=1)):
        m = Model(2, 2, 4, seed=8, **kw)
        sh = m.gpu.shape
        cache = kivi.KiviCache(sh)
        m.chunk([150, 150], pad=0)
        x = m.dev
        k, v = (t.unflatten(0, (2, 150)).transpose(1, 2).contiguous() for t in (x["k"], x["v"]))
        cache.quantize_prefill(k, v)
        m.gpu.append(x["k"], x["v"], x["offsets"], 150)
        m.append()
        view = paged.KiviPagedCache.from_cache(cache)
        m.chunk([1, 1], pad=0)
        q = m.dev["q"].contiguous()
        off = m.dev["offsets"]
        a = view.attention(q, offsets=off, max_new=1)
        b = m.gpu.attention(q, offsets=off, max_new=1)
        assert torch.equal(a, b)                       # where pages lie does not matter
        want, tol = m.attention(new=False)
        close(a, want, tol, "paged view")
        ref = cache.decode_attention(q)
        assert ((ref.double().cpu() - want).abs().amax(-1) <= 2e-3 * want.abs().amax(-1)).all()


def test_a_workspace_of_nan_patterns_changes_nothing():
    """Nothing is read from the workspace that the call did not write there."""
    for kw in (dict(), dict(bits=4, G=16, R=32), dict(bits=8, G=32, R=64, fp8=1)):
        m = Model(3, 2, 4, seed=18, max_new=90, columns=40, **kw)
        fill(m, [0, 333, 500])
        assert m.gpu.status() == 0
        for counts in ([1, 0, 1], [3, 16, 1], [90, 1, 0]):
            m.chunk(counts)
            m.gpu.workspace.fill_(0xff)
            attend(m)
            m.gpu.workspace.fill_(0xff)
            w, x = torch.zeros((6, m.columns), device="cuda"), m.dev
            m.gpu.weights(w, x["q"], x["k"], x["offsets"], x["max_new"])
            close(w, *m.weights(), "weights")


@pytest.mark.parametrize("cap", [1e4, 1e7, 1e25])
def test_a_large_cap_keeps_the_scores(cap):
    """Scores far below the cap: c tanh(s / c) is s (1 - (s/c)^2 / 3), which the
    kernels hold to 2^-20 of the score, inside the bound's share of a score's
    size without the cap's own term.  |s| < 100 here: p differs from the
    uncapped one by less than 2 100^3 / 3e8 < 1 %, and the bound, which is
    proportional to it, by as little."""
    for counts in ([1], [9], [70]):
        m = Model(1, 2, 4, seed=19, max_new=70, columns=24)
        fill(m, [444])
        m.chunk(counts)
        x, n = m.dev, counts[0]
        want, _ = m.attention(cap)
        plain, tol = m.attention(0.0)
        out = m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], n, softcap=cap)
        close(out[:n], want, tol * 1.01, f"{counts}")
        w = m.gpu.weights(torch.zeros((2, m.columns), device="cuda"), x["q"], x["k"], x["offsets"], n, softcap=cap)
        close(w, m.weights(cap)[0], m.weights(0.0)[1] * 1.01, f"weights {counts}")


@pytest.mark.parametrize("kw", [dict(bits=4, G=64, R=64), dict(bits=2, G=32, R=64), dict(bits=4, G=16, R=32, meta=1)])
@pytest.mark.parametrize("counts,small", [([1, 1], -8), ([9, 2], -8), ([70, 33], -16)])
def test_small_numbers(kw, counts, small):
    """Keys near 2^-13 under queries near 2^12 and small values: scales below
    fp16's normal numbers.  Beside the bound of `attention`: a key is carried
    halved, so fp16's fixed step leaves 2^-24 of it, sum_c |q_c| tau 2^-24 of a
    score; few query rows round p s to fp16, 2^-25 at least, which multiplies
    |code - z| <= 2^bits - 1 (groups that span zero), per token seen and divided
    by the sum of the p, which is one over the largest normalised p."""
    m = Model(2, 2, 4, seed=25, max_new=70, columns=48, **kw)
    scales = (2.0 ** 12, 2.0 ** -13, 2.0 ** small)
    x = m.chunk([400, 333], scales=scales)
    m.gpu.append(x["k"], x["v"], x["offsets"], x["max_new"])
    m.append()
    assert m.gpu.status() == 0
    x = m.chunk(counts, scales=scales)
    n = sum(counts)
    out = m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], max(counts))
    want, tol = m.attention()
    step = torch.expm1(2 * 2.0 ** -24 * m.q[:n].double().abs().sum(-1, keepdim=True) / 128 ** 0.5)
    for b in range(2):
        sl = slice(m.off[b], m.off[b + 1])
        for i in range(8):
            K, V, cached, _ = m.keys(b, i // 4)
            p, _ = m.softmax(b, i, K, cached, 0.0, True)
            tol[sl, i] += 2 * step[sl, i] * V.abs().max()
            if max(counts) * 4 <= 64:
                tol[sl, i] += 2.0 ** -25 * (2 ** kw["bits"] - 1) * K.shape[0] * p.amax(1, keepdim=True)
    close(out[:n], want, tol, "attention")
    w = m.gpu.weights(torch.zeros((4, m.columns), device="cuda"), x["q"], x["k"], x["offsets"], max(counts))
    # many rows carry halved keys here too: their low parts end at the same 2^-24
    want, tol = m.weights()
    close(w, want, tol + (float(step.max()) * want if max(counts) * 4 > 64 or kw["G"] == 16 else 0.0), "weights")


def test_captured_long_chunks_share_a_workspace():
    """Two caches, one workspace: a graph of each one's long chunk, replayed in
    turn over growing caches; every replay sees its own."""
    ms = [Model(2, 2, 4, seed=20 + i, max_new=80, columns=16, R=32) for i in range(2)]
    ws = ms[0].gpu.workspace
    caches = [paged.KiviPagedCache(m.gpu.shape, m.num_pages, 80, buffers=(
        m.gpu.pool, m.gpu.k_fp16, m.gpu.v_fp16, m.gpu.table, m.gpu.n_tokens, m.gpu.n_evicted), workspace=ws) for m in ms]
    runs, offsets = [], []                        # a graph reads its offsets again at every replay
    side = torch.cuda.Stream()
    for m, c in zip(ms, caches):
        fill(m, [70, 5])
        x = m.chunk([80, 21], pad=0)
        q, k, v, off = x["q"].clone(), x["k"].clone(), x["v"].clone(), x["offsets"].clone()
        out, w = torch.zeros_like(q), torch.zeros((4, m.columns), device="cuda")
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            c.attention(q, k, v, off, 80, out=out)
            w.zero_()
            c.weights(w, q, k, off, 80)
        torch.cuda.current_stream().wait_stream(side)
        runs.append((m, g, q, k, v, out, w))
        offsets.append(off)
    for i in range(3):
        for m, g, q, k, v, out, w in runs:
            x = m.chunk([80, 21], pad=0)
            for t, name in ((q, "q"), (k, "k"), (v, "v")):
                t.copy_(x[name])
        for m, g, q, k, v, out, w in runs + runs:
            g.replay()
        for m, g, q, k, v, out, w in runs:
            close(out, *m.attention(), f"replay {i}")
            close(w, *m.weights(), f"weights {i}")
            fill(m, [33, 40])


def test_pairs_in_several_launches():
    """A table so long that its tiles do not fit the workspace at once: the
    pairs are staged and worked on in two launches."""
    m = Model(4, 4, 1, seed=22, max_new=80, columns=4096)
    fill(m, [300, 0, 77, 1])
    m.chunk([80, 65, 1, 70])
    n = m.gpu.kernel_launches
    attend(m)
    assert m.gpu.kernel_launches - n == 8
    x = m.dev
    w = m.gpu.weights(torch.zeros((16, m.columns), device="cuda"), x["q"], x["k"], x["offsets"], x["max_new"])
    close(w, *m.weights(), "weights")


def test_weights_of_many_rows_in_several_launches():
    """Page sums of all query rows at once would be too large: eight tiles of
    256 rows go in launches of fewer."""
    m = Model(1, 1, 1, seed=23, max_new=2048, columns=40960)
    fill(m, [200])
    m.chunk([2048])
    x = m.dev
    n = m.gpu.kernel_launches
    w = m.gpu.weights(torch.zeros((1, m.columns), device="cuda"), x["q"], x["k"], x["offsets"], 2048, max_cached=256)
    assert m.gpu.kernel_launches - n > 3
    close(w, *m.weights(), "weights")


# ------------------------------------------------------------------- evict ---

def random_weights(gen, P, C, kind):
    w = torch.rand((P, C), generator=gen) ** 6
    if kind == "ties":
        w = (w * 4).floor() / 4
    if kind == "odd":
        w[:, ::3] = float("nan")
        w[:, 1::5] = float("inf")
        w[:, 2::7] = float("-inf")
        w[:, 3::4] = -0.0
        w[:, 4::9] = 0.0
        w[:, 5::6] *= -1e-40
    return w


@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
@pytest.mark.parametrize("held,budget,recent", [(1, 0, 0), (7, 3, 1), (40, 40, 3), (40, 39, 0), (40, 1, 5),
                                                (1025, 1024, 8), (2500, 700, 33), (2500, 1, 0), (2500, 2499, 2499)])
def test_evict_is_a_stable_selection(kind, held, budget, recent):
    B, H, R, G = 2, 3, 32, 32
    P, C = B * H, held + 4
    gen = torch.Generator().manual_seed(held + budget)
    n = [held, max(held - 2, 0)]
    shape = kivi.CacheShape(2, G, R, B, H, H, 128, C * G)
    c = paged.KiviPagedCache(shape)
    c.n_tokens.copy_(torch.tensor([x * G + 1 for x in n]))
    table = torch.randperm(P * C, generator=gen).view(P, C).int()
    c.table.copy_(table)
    w0 = random_weights(gen, P, C, kind)
    w = w0.cuda()
    c.evict(w, budget, recent)
    got_t, got_w = c.table.cpu(), w.cpu()
    for p in range(P):
        np_ = n[p // H]
        want_t, want_w = table[p].clone(), w0[p].clone()
        if np_ > budget:
            keep, drop = pick(w0[p, :np_].tolist(), budget, recent)
            want_t[:np_] = table[p][keep + drop]
            want_w[:np_] = torch.cat([w0[p][keep], torch.zeros(len(drop))])
        assert torch.equal(got_t[p], want_t), f"table of pair {p}"
        assert torch.equal(got_w[p].view(torch.int32), want_w.view(torch.int32)), f"weights of pair {p}"
    assert c.n_evicted.tolist() == [max(0, x - budget) for x in n]
    assert c.status() == 0
    before = c.table.clone()
    c.evict(w, budget, recent)                        # nothing left to evict
    assert torch.equal(before, c.table) and c.n_evicted.tolist() == [max(0, x - budget) for x in n]


# --------------------------------------------------------------- together ---

@pytest.mark.parametrize("kw", [dict(bits=2, G=32, R=64, sink=4, columns=12),
                                dict(bits=4, G=16, R=32, flush=1, columns=24),
                                dict(bits=8, G=32, R=32, fp8=1, columns=12)])
def test_a_serving_run(kw):
    """Prompt chunks, decode steps whose weights add up, evictions, more
    tokens into the freed pages: attention, weights, table and records agree
    with the model all along."""
    m = Model(3, 2, 4, seed=9, max_new=150, **kw)
    w = torch.zeros((6, m.columns), device="cuda")
    total = torch.zeros((6, m.columns), dtype=torch.float64)
    for step in range(5):
        for counts in ([150, 40, 0], [1, 1, 1], [3, 1, 20]):
            x = m.chunk(counts)
            attend(m, max_cached=m.columns * m.G + m.sink + m.R)
            before = w.clone()
            m.gpu.weights(w, x["q"], x["k"], x["offsets"], x["max_new"])
            close(w, *m.weights(base=before.cpu()), "weights")
            m.gpu.append(x["k"], x["v"], x["offsets"], x["max_new"])
            m.append()
            m.check_state()
        want_t, want_w = m.evict(m.gpu.table.cpu().numpy(), w.cpu().numpy(), 4, 2)
        m.gpu.evict(w, 4, 2)
        assert np.array_equal(m.gpu.table.cpu().numpy(), want_t)
        assert np.array_equal(w.cpu().numpy(), want_w)
        m.check_state()
    assert max(m.gpu.n_evicted.tolist()) > 8


def test_captured_steps_follow_the_lengths():
    """One graph of (attention, weights, append, evict), replayed: it sees the
    sequences grow and lose pages; a second graph shares its workspace."""
    m = Model(2, 2, 4, seed=10, max_new=8, columns=8, R=32)
    fill(m, [100, 31])
    x = m.chunk([2, 1], pad=0)
    bufs = {k: x[k].clone() for k in ("q", "k", "v")}
    off = x["offsets"].clone()
    w = torch.zeros((4, m.columns), device="cuda")
    out = torch.zeros_like(bufs["q"])
    side = torch.cuda.Stream()

    def step():
        m.gpu.attention(bufs["q"], bufs["k"], bufs["v"], off, 2, out=out)
        m.gpu.weights(w, bufs["q"], bufs["k"], off, 2)
        m.gpu.append(bufs["k"], bufs["v"], off, 2)

    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g1, stream=side):
            step()
        with torch.cuda.graph(g2, stream=side):
            m.gpu.evict(w, 4, 1)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(60):
        x = m.chunk([2, 1], pad=0)
        for k in bufs:
            bufs[k].copy_(x[k])
        want, tol = m.attention()
        g1.replay()
        close(out, want, tol, f"replay {i}")
        m.append()
        if i % 7 == 6:
            want_t, want_w = m.evict(m.gpu.table.cpu().numpy(), w.cpu().numpy(), 4, 1)
            g2.replay()
            assert np.array_equal(m.gpu.table.cpu().numpy(), want_t)
            assert np.array_equal(w.cpu().numpy(), want_w)
        m.check_state()


def test_other_streams_and_equal_bits():
    """Calls on a stream that is not current give the same bits as on the
    current one, twice."""
    m = Model(2, 2, 4, seed=11, max_new=40, columns=40)
    fill(m, [900, 300])
    x = m.chunk([40, 7])
    a = m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], 40)
    wa = m.gpu.weights(torch.zeros((4, m.columns), device="cuda"), x["q"], x["k"], x["offsets"], 40)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    wb = torch.zeros((4, m.columns), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    b = m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], 40, stream=s)
    m.gpu.weights(wb, x["q"], x["k"], x["offsets"], 40, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a[:47], b[:47]) and torch.equal(wa, wb)


def test_two_caches_on_two_streams_at_once():
    """Calls of two caches with workspaces of their own, enqueued in turn on two
    streams without waiting, give the bits they give one after the other."""
    ms = [Model(2, 2, 4, seed=30 + i, max_new=80, columns=24) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ms]
    for m in ms:
        fill(m, [333, 500])
    for counts in ([80, 33], [1, 1], [7, 3]):
        xs = [m.chunk(counts, pad=0) for m in ms]
        refs = []
        for m, x in zip(ms, xs):
            w = m.gpu.weights(torch.zeros((4, m.columns), device="cuda"), x["q"], x["k"], x["offsets"], x["max_new"])
            refs.append((m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], x["max_new"]), w))
        outs = [[torch.zeros_like(a) for _ in range(8)] for a, _ in refs]
        ws = [[torch.zeros_like(w) for _ in range(8)] for _, w in refs]
        torch.cuda.synchronize()
        for i in range(8):
            for j, (m, x, s) in enumerate(zip(ms, xs, streams)):
                m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], x["max_new"], out=outs[j][i], stream=s)
                m.gpu.weights(ws[j][i], x["q"], x["k"], x["offsets"], x["max_new"], stream=s)
        torch.cuda.synchronize()
        for j, (a, w) in enumerate(refs):
            assert all(torch.equal(o, a) for o in outs[j]) and all(torch.equal(o, w) for o in ws[j])


def test_pool_offsets_pass_32_bits():
    """Pages beyond the first 4 GB of a pool, written and read."""
    m = Model(1, 2, 2, seed=12)
    n = (5 << 30) // m.gpu.pool.shape[1]
    shape, P = m.gpu.shape, 2
    pool = torch.empty((n, m.gpu.pool.shape[1]), dtype=torch.uint8, device="cuda")
    table = (n - 1 - torch.arange(P * m.columns, dtype=torch.int32)).view(P, -1).cuda()
    big = paged.KiviPagedCache(shape, n, max_new=8, buffers=(pool, torch.empty_like(m.gpu.k_fp16),
                               torch.empty_like(m.gpu.v_fp16), table, torch.zeros(1, dtype=torch.int32, device="cuda"),
                               torch.zeros(1, dtype=torch.int32, device="cuda")))
    for counts in ([300], [70]):
        x = m.chunk(counts)
        for c in (m.gpu, big):
            c.append(x["k"], x["v"], x["offsets"], x["max_new"])
        m.append()
    x = m.chunk([8])
    outs = [c.attention(x["q"], x["k"], x["v"], x["offsets"], 8)[:8] for c in (m.gpu, big)]
    assert torch.equal(*outs)
    close(outs[0], *m.attention(), "attention")


# ------------------------------------------------- what the device refuses ---

def test_bad_pages_are_reported_and_harm_no_other_sequence():
    m = Model(2, 2, 4, seed=13, max_new=20)
    fill(m, [200, 200])
    x = m.chunk([20, 20])
    want, tol = m.attention()
    good = m.gpu.table.clone()
    for bad in (-1, m.num_pages, 2 ** 31 - 1):
        m.gpu.table.copy_(good)
        m.gpu.table[0, 1] = bad                       # sequence 0, kv head 0
        m.gpu.control.zero_()
        out = m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], 20)
        w = m.gpu.weights(torch.zeros((4, m.columns), device="cuda"), x["q"], x["k"], x["offsets"], 20)
        assert m.gpu.status() == kivi.KIVI_STATUS_BAD_PAGE
        close(out[20:40], want[20:], tol[20:], "the other sequence")
        assert torch.isfinite(w).all()
        # an append whose next page is not one of the pool's
        m.gpu.control.zero_()
        m.gpu.table.copy_(good)
        m.gpu.table[0, 6] = bad                       # column 6 is the next free one of 200 tokens
        pool = m.gpu.pool.clone()
        tokens = m.gpu.n_tokens.clone()
        y = {k: x[k].repeat(4, 1, 1) for k in ("k", "v")}
        rows = [t.clone() for t in (m.gpu.k_fp16, m.gpu.v_fp16)]
        m.gpu.append(y["k"], y["v"], torch.tensor([0, 80, 80], dtype=torch.int32, device="cuda"), 80)
        assert m.gpu.status() == kivi.KIVI_STATUS_BAD_PAGE
        changed = (m.gpu.pool != pool).any(1).nonzero().flatten().tolist()
        assert set(changed) <= set(good[0, 6:].tolist() + good[1, 6:].tolist())
        for t, r in zip((m.gpu.pool, m.gpu.n_tokens, m.gpu.k_fp16, m.gpu.v_fp16), (pool, tokens, *rows)):
            t.copy_(r)
    m.gpu.table.copy_(good)
    m.gpu.control.zero_()
    m.check_state()


def test_bad_lengths_skip_their_sequence_alone():
    m = Model(3, 1, 2, seed=14, max_new=10)
    fill(m, [100, 100, 100])
    x = m.chunk([10, 10, 10], pad=0)
    want, tol = m.attention()
    tokens, gone = m.gpu.n_tokens.clone(), m.gpu.n_evicted.clone()
    off = x["offsets"]

    def offsets(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    cases = [(None, None, offsets(0, 10, 9, 30), [0]),       # descending, then 21 tokens
             (None, None, offsets(-1, 10, 20, 30), [1, 2]),
             (None, None, offsets(0, 10, 20, 31), [0, 1]),
             ((1, -1), None, off, [0, 2]), ((0, 2 ** 31 - 1), None, off, [1, 2]),
             (None, (2, -1), off, [0, 1]), (None, (2, 99), off, [0, 1])]
    for tok, ev, o, fine in cases:
        m.gpu.control.zero_()
        m.gpu.n_tokens.copy_(tokens)
        m.gpu.n_evicted.copy_(gone)
        if tok:
            m.gpu.n_tokens[tok[0]] = tok[1]
        if ev:
            m.gpu.n_evicted[ev[0]] = ev[1]
        state = [t.clone() for t in (m.gpu.pool, m.gpu.k_fp16, m.gpu.v_fp16, m.gpu.n_tokens)]
        out = torch.full_like(x["q"].contiguous(), 7.0)
        m.gpu.attention(x["q"], x["k"], x["v"], o, 10, out=out)
        assert m.gpu.status() == kivi.KIVI_STATUS_BAD_STATE
        for b in range(3):
            if b in fine:
                close(out[10 * b:10 * b + 10], want[10 * b:10 * b + 10], tol[10 * b:10 * b + 10], f"sequence {b}")
        touched = sorted({i for b in fine for i in range(10 * b, 10 * b + 10)})
        rest = [i for i in range(30) if i not in touched]
        assert (out[rest] == 7.0).all()
        w = torch.zeros((3, m.columns), device="cuda")
        m.gpu.weights(w, x["q"], x["k"], o, 10)
        assert all((w[b] == 0).all() for b in range(3) if b not in fine)
        m.gpu.append(x["k"], x["v"], o, 10)
        grown = m.gpu.n_tokens - state[3]
        assert [b for b in range(3) if grown[b]] == fine
        for t, s in zip((m.gpu.pool, m.gpu.k_fp16, m.gpu.v_fp16), state):
            t.copy_(s)
    # more cached tokens than max_cached says, in every sequence
    m.gpu.n_tokens.copy_(tokens)
    m.gpu.n_evicted.copy_(gone)
    m.gpu.control.zero_()
    out = torch.full_like(x["q"].contiguous(), 7.0)
    m.gpu.attention(x["q"], x["k"], x["v"], off, 10, max_cached=99, out=out)
    assert (out == 7.0).all() and m.gpu.status() == kivi.KIVI_STATUS_BAD_STATE
    # more new tokens than max_new says, in every sequence
    m.gpu.n_tokens.copy_(tokens)
    m.gpu.n_evicted.copy_(gone)
    m.gpu.control.zero_()
    out = torch.full_like(x["q"].contiguous(), 7.0)
    m.gpu.attention(x["q"], x["k"], x["v"], off, 9, out=out)
    m.gpu.append(x["k"], x["v"], off, 9)
    assert (out == 7.0).all() and torch.equal(m.gpu.n_tokens, tokens)
    assert m.gpu.status() == kivi.KIVI_STATUS_BAD_STATE


def test_an_append_beyond_the_table_is_refused():
    m = Model(2, 1, 1, seed=15, columns=4, R=32)             # 4 pages of 32 tokens
    fill(m, [129, 20])                                       # full: 4 pages and one token
    m.check_state()
    fill(m, [31, 1])                                         # the window takes 31 more
    m.check_state()
    x = m.chunk([1, 5])
    before = [t.clone() for t in (m.gpu.pool, m.gpu.k_fp16[:1], m.gpu.v_fp16[:1])]
    m.gpu.append(x["k"], x["v"], x["offsets"], 5)
    assert m.gpu.status() == kivi.KIVI_STATUS_CAPACITY
    assert m.gpu.n_tokens.tolist() == [160, 26]
    for t, s in zip((m.gpu.pool, m.gpu.k_fp16[:1], m.gpu.v_fp16[:1]), before):
        assert torch.equal(t.view(torch.uint8), s.view(torch.uint8))
    # evicting makes room
    m.gpu.control.zero_()
    m.gpu.evict(torch.rand((2, 4), device="cuda"), 3)
    m.gpu.append(x["k"][:1], x["v"][:1], torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda"), 1)
    assert m.gpu.status() == 0 and m.gpu.n_tokens.tolist() == [161, 26] and m.gpu.n_evicted.tolist() == [1, 0]


def test_nothing_to_do_is_no_launch():
    m = Model(2, 1, 2, seed=16)
    q = torch.empty((0, 2, 128), dtype=torch.float16, device="cuda")
    kv = torch.empty((0, 1, 128), dtype=torch.float16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    n = m.gpu.kernel_launches
    assert m.gpu.attention(q, kv, kv, off).shape == (0, 2, 128)
    m.gpu.append(kv, kv, off)
    m.gpu.weights(torch.zeros((2, m.columns), device="cuda"), q, kv, off)
    assert m.gpu.kernel_launches == n
    # all sequences empty, but rows to spare
    m.chunk([0, 0], pad=4)
    x = m.dev
    out = torch.full((4, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], 1, out=out)
    m.gpu.append(x["k"], x["v"], x["offsets"], 1)
    assert (out == 7.0).all() and m.gpu.n_tokens.tolist() == [0, 0] and m.gpu.status() == 0


def test_a_longer_chunk_than_the_workspace_is_refused():
    m = Model(1, 1, 4, seed=17, max_new=2)
    x = m.chunk([2000])
    with pytest.raises(kivi.KiviError) as e:
        m.gpu.attention(x["q"], x["k"], x["v"], x["offsets"], 2000)
    assert e.value.status == kivi.KIVI_ERR_WORKSPACE
