"""The paged latent cache's operators against plain 64-bit forms (B200).

Tolerances, derived from the number of roundings (bf16 rounds by at most u =
2^-8 of the value, fp32 by 2^-24):

  attention  the probabilities are rounded to bf16 and the output is: at most
             u (|out| + A) with A = sum_j softmax_j |c_j|; a logit of dk fp32
             products summed in fp32 is off by at most X = (dk + 8) 2^-24
             scale sum |q c| (8: scaling, the subtraction of the maximum and the
             exponential), which moves each probability by X and their sum by
             X: 2 X A; lse by X and its own rounding.
  rotation   the angle is off by at most pi 2^-24 and cosine, sine and scale
             by a few ulps, the two products and the sum by three: together
             under 2^-20 of the pair's length; then one rounding to the type.
  page moves exact.
"""
import itertools
import threading

import pytest
import torch

import gated_delta_rule_88_b200 as kda
from gated_delta_rule_88_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Cache:
    """A paged cache with N sequences of the given lengths; rows that hold no
    key, unused pages and the table's padding are poisoned."""

    def __init__(self, lens, page, dk, seed=0, spare=3, poison=float("nan"), pad=-1, gap=0, dtype=torch.bfloat16):
        g = gen(seed)
        per = [-(-n // page) for n in lens]
        total = sum(per) + spare
        ids = torch.randperm(total, generator=g)
        self.table = torch.full((len(lens), max(1, *per) if len(per) > 1 else max(1, per[0])), pad, dtype=torch.int32)
        stride = page * dk + gap
        self.flat = torch.full((total * stride + 8,), poison, dtype=dtype)
        self.cache = self.flat[:total * stride].view(total, stride)[:, :page * dk].view(total, page, dk) if gap else \
            self.flat[:total * stride].view(total, page, dk)
        self.keys = []
        k = 0
        for n, m in enumerate(lens):
            x = torch.randn(m, dk, generator=g).to(dtype)
            self.keys.append(x)
            for j in range(per[n]):
                self.table[n, j] = ids[k]
                rows = x[j * page:(j + 1) * page]
                self.cache[ids[k], :len(rows)] = rows
                k += 1
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.gap = gap

    def to_gpu(self):
        flat = self.flat.to(DEV)
        total, page, dk = self.cache.shape
        stride = page * dk + self.gap
        c = flat[:total * stride].view(total, stride)[:, :page * dk].unflatten(1, (page, dk))
        return c, self.table.to(DEV), self.lens.to(DEV)


def oracle(q, keys, counts, dv, scale, causal=True):
    """out, lse, and the bounds of their errors, in 64 bits."""
    T, H, dk = q.shape
    out = torch.zeros(T, H, dv, dtype=torch.float64)
    lse = torch.full((T, H), -float("inf"), dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    t = 0
    for n, count in enumerate(counts):
        k = keys[n].double()
        for i in range(count):
            see = max(0, len(k) - count + i + 1) if causal else len(k)
            if see:
                x = q[t].double() @ k[:see].T * scale
                p = torch.softmax(x, -1)
                out[t] = p @ k[:see, :dv]
                lse[t] = torch.logsumexp(x, -1)
                size = abs(scale) * (q[t].double().abs() @ k[:see].abs().T).amax(-1)
                X = ((dk + 8) * 2.0 ** -24 * size + 2.0 ** -22)[:, None]
                A = p @ k[:see, :dv].abs()
                tol[t] = U * (out[t].abs() + A) * (1 + 2 * U) + 2 * X * A + 1e-30
                ltol[t] = X[:, 0] + 2.0 ** -22 * (1 + lse[t].abs())
            t += 1
    return out, lse, tol, ltol


def check_attn(out, lse, ref, rows=None):
    o, l, tol, ltol = ref
    sel = slice(None) if rows is None else rows
    out, lse = out.double().cpu()[sel], lse.double().cpu()[sel]
    o, l, tol, ltol = o[sel], l[sel], tol[sel], ltol[sel]
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert (out[empty] == 0).all()
    bad = (out - o).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} outputs off, first at {torch.nonzero(bad)[0].tolist()}, worst " \
                          f"{float(((out - o).abs() / tol.clamp_min(1e-30)).max()):.2f} x the bound"
    lbad = ((lse - l).abs() > ltol) & ~empty
    assert not lbad.any(), f"{int(lbad.sum())} lse off, worst {float(((lse - l).abs() / ltol)[~empty].max()):.2f} x the bound"


def run_attn(c, counts, H, dv, seed=1, causal=True, varlen=None, scale=None, qscale=1.0, extra=0):
    dk = c.cache.shape[2]
    T = sum(counts)
    q = (torch.randn(T + extra, H, dk, generator=gen(seed)) * qscale).to(torch.bfloat16)
    varlen = len(set(counts)) > 1 if varlen is None else varlen
    cu = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32, device=DEV) if varlen or extra else None
    cache, table, lens = c.to_gpu()
    scale = 0.0722 if scale is None else scale
    out = torch.full((T + extra, H, dv), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + extra, H), 7.0, device=DEV)
    kda.kda_latent_attn(q.to(DEV), cache, table, lens, dv=dv, cu_seqlens=cu, out=out, lse=lse, scale=scale, causal=causal)
    torch.cuda.synchronize()
    return q, out, lse, scale


@pytest.mark.parametrize("lens,counts,H,page,dv,dr", [
    ([1], [1], 1, 16, 512, 64),
    ([1], [1], 32, 64, 512, 64),
    ([2, 1], [1, 1], 16, 64, 512, 64),
    ([127, 128, 129], [1, 1, 1], 32, 64, 512, 64),
    ([300], [1], 32, 64, 512, 64),
    ([300, 17, 999], [1, 1, 1], 20, 16, 512, 64),
    ([500, 40], [1, 1], 64, 128, 512, 64),
    ([500, 40], [1, 1], 128, 32, 512, 0),
    ([500, 40], [1, 1], 33, 32, 256, 0),
    ([257, 511], [1, 1], 48, 32, 256, 64),
    ([640], [4], 32, 64, 512, 64),
    ([130, 5], [2, 2], 16, 16, 512, 64),
    ([130, 260], [3, 3], 33, 64, 512, 64),
    ([70, 200, 33], [70, 1, 5], 16, 16, 512, 64),
    ([1000, 3], [9, 3], 7, 64, 256, 64),
    ([4000], [1], 8, 128, 512, 64),
    ([1500, 1], [2, 1], 3, 16, 512, 0),
    ([129] * 40, [1] * 40, 32, 64, 512, 64),
])
def test_attn_matches_the_formula(lens, counts, H, page, dv, dr):
    c = Cache(lens, page, dv + dr, seed=len(lens) + H)
    q, out, lse, scale = run_attn(c, counts, H, dv)
    assert kda.kda_get_device_error() == 0
    check_attn(out, lse, oracle(q, c.keys, counts, dv, scale))


@pytest.mark.parametrize("causal", [True, False])
def test_attn_rows_that_see_nothing(causal):
    """Empty caches, and new tokens before the first cached key."""
    lens, counts = [0, 2, 5, 0], [3, 5, 5, 1]
    c = Cache(lens, 16, 576, seed=3)
    q, out, lse, scale = run_attn(c, counts, 32, 512, causal=causal)
    assert kda.kda_get_device_error() == 0
    check_attn(out, lse, oracle(q, c.keys, counts, 512, scale, causal))


def test_attn_without_the_causal_mask():
    c = Cache([200, 31], 32, 576, seed=4)
    q, out, lse, scale = run_attn(c, [40, 40], 16, 512, causal=False)
    check_attn(out, lse, oracle(q, c.keys, [40, 40], 512, scale, causal=False))


@pytest.mark.parametrize("pad", [-1, 1 << 30])
def test_attn_never_uses_what_lies_behind_the_keys(pad):
    """The table's padding, unused pages and the rest of the last page hold
    anything (infinities and NaN here)."""
    for poison in (float("inf"), -float("inf"), float("nan")):
        c = Cache([65, 1, 200], 64, 576, seed=5, poison=poison, pad=pad)
        q, out, lse, scale = run_attn(c, [1, 1, 1], 32, 512)
        assert kda.kda_get_device_error() == 0
        check_attn(out, lse, oracle(q, c.keys, [1, 1, 1], 512, scale))


def test_attn_rows_behind_the_last_sequence_stay():
    c = Cache([50, 60], 16, 576, seed=6)
    q, out, lse, scale = run_attn(c, [2, 3], 32, 512, extra=4)
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()
    ref = oracle(q[:5], c.keys, [2, 3], 512, scale)
    check_attn(out[:5], lse[:5], ref)


def test_attn_empty_sequences_among_others():
    c = Cache([50, 9, 60, 5], 16, 576, seed=16)
    q, out, lse, scale = run_attn(c, [0, 2, 0, 3], 32, 512)
    check_attn(out, lse, oracle(q, c.keys, [0, 2, 0, 3], 512, scale))


def test_attn_steep_and_flat_logits():
    """One key dominates (the maximum jumps between tiles) or all weigh alike."""
    for qscale in (40.0, 0.0, 1e-3):
        c = Cache([700, 130], 64, 576, seed=7)
        q, out, lse, scale = run_attn(c, [1, 1], 32, 512, qscale=qscale)
        check_attn(out, lse, oracle(q, c.keys, [1, 1], 512, scale))


@pytest.mark.parametrize("scale", [-0.05, 0.0])
def test_attn_any_finite_scale(scale):
    c = Cache([300], 64, 576, seed=8)
    q, out, lse, _ = run_attn(c, [2], 32, 512, scale=scale)
    check_attn(out, lse, oracle(q, c.keys, [2], 512, scale))


def test_attn_growing_maximum():
    """Keys of increasing size: the running maximum is raised in every tile."""
    c = Cache([1200], 64, 576, seed=9)
    ramp = torch.linspace(0.05, 6, 1200)[:, None]
    c.keys[0] = (c.keys[0].float() * ramp).to(torch.bfloat16)
    for j in range(c.table.shape[1]):
        rows = c.keys[0][64 * j:64 * j + 64]
        c.cache[c.table[0, j], :len(rows)] = rows
    q, out, lse, scale = run_attn(c, [3], 32, 512)
    check_attn(out, lse, oracle(q, c.keys, [3], 512, scale))


def test_attn_strided_and_shared_pages():
    """Pages of several layers side by side (only one layer is read), and one
    page in two sequences' tables."""
    c = Cache([64, 128, 70], 64, 576, seed=10, gap=64 * 576 * 2)
    c.table[1, 0] = c.table[0, 0]
    c.keys[1] = torch.cat([c.keys[0], c.keys[1][64:]])
    q, out, lse, scale = run_attn(c, [1, 1, 1], 32, 512)
    check_attn(out, lse, oracle(q, c.keys, [1, 1, 1], 512, scale))


def test_attn_offsets_past_32_bits():
    """Pages 2^26 elements apart: the last ones lie beyond 2^32 bytes."""
    pages, page, dk, H = 70, 16, 576, 16
    flat = torch.empty((pages - 1) * (1 << 26) + page * dk, dtype=torch.bfloat16, device=DEV)
    cache = flat.as_strided((pages, page, dk), (1 << 26, dk, 1))
    keys = torch.randn(40, dk, generator=gen(11)).to(torch.bfloat16)
    ids = [69, 0, 68]
    for j, i in enumerate(ids):
        rows = keys[16 * j:16 * j + 16]
        cache[i, :len(rows)] = rows.to(DEV)
    table = torch.tensor([ids], dtype=torch.int32, device=DEV)
    q = torch.randn(1, H, dk, generator=gen(12)).to(torch.bfloat16)
    out, lse = kda.kda_latent_attn(q.to(DEV), cache, table, torch.tensor([40], dtype=torch.int32, device=DEV), scale=0.07)
    check_attn(out, lse, oracle(q, [keys], [1], 512, 0.07))
    # and the write to them
    new = torch.randn(40, dk, generator=gen(13)).to(torch.bfloat16).to(DEV)
    kda.kda_latent_append(new, cache, table, torch.tensor([40], dtype=torch.int32, device=DEV))
    assert torch.equal(torch.cat([cache[69], cache[0], cache[68]])[:40], new)


@pytest.mark.parametrize("how", ["page", "negative page", "long", "negative"])
def test_attn_bad_sequences_are_reported_and_not_written(how):
    c = Cache([100, 300, 50], 16, 576, seed=14)
    if how == "page":
        c.table[1, 17] = c.cache.shape[0]
    elif how == "negative page":
        c.table[1, 0] = -1
    elif how == "long":
        c.lens[1] = c.table.shape[1] * 16 + 1
    else:
        c.lens[1] = -1
    q, out, lse, scale = run_attn(c, [2, 2, 2], 32, 512)
    assert kda.kda_get_device_error() == 5
    assert (out[2:4] == 7).all() and (lse[2:4] == 7).all()
    check_attn(out, lse, oracle(q, c.keys, [2, 2, 2], 512, scale), rows=[0, 1, 4, 5])


def test_attn_same_bits_every_time_on_any_stream_and_without_lse():
    c = Cache([3000, 700, 5], 64, 576, seed=15)
    q, out, lse, scale = run_attn(c, [3, 3, 3], 32, 512)
    cache, table, lens = c.to_gpu()
    qd = q.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out2, lse2 = kda.kda_latent_attn(qd, cache, table, lens, scale=scale)
    s.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    out3 = torch.empty_like(out)
    lib = kda.load_library()
    rc = lib.kda_latent_attn(qd.data_ptr(), cache.data_ptr(), table.data_ptr(), lens.data_ptr(), None, out3.data_ptr(),
                             None, 9, 32, 576, 512, 3, cache.shape[0], 64, table.shape[1], 0, scale, 0, 1, None)
    assert rc == 0
    torch.cuda.synchronize()
    assert torch.equal(out, out3)


def test_attn_two_graphs_replayed_side_by_side():
    """Two captured calls, replayed on two streams at once, and eager calls
    between them: each has a workspace of its own."""
    cases = []
    for seed, lens in ((20, [2000, 300]), (21, [900, 1400])):
        c = Cache(lens, 64, 576, seed=seed)
        q, out, lse, scale = run_attn(c, [1, 1], 32, 512, seed=seed)
        cache, table, ln = c.to_gpu()
        qd, og, lg = q.to(DEV), torch.zeros_like(out), torch.zeros_like(lse)
        call = lambda og=None, lg=None, qd=qd, cache=cache, table=table, ln=ln, scale=scale: kda.kda_latent_attn(
            qd, cache, table, ln, out=og, lse=lg, scale=scale)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(og, lg)
        cases.append((graph, torch.cuda.Stream(), og, lg, out, lse, call))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, *_ in cases:
            with torch.cuda.stream(stream):
                graph.replay()
        eager = cases[0][6]()
    torch.cuda.synchronize()
    assert kda.kda_get_device_error() == 0
    assert torch.equal(eager[0], cases[0][4])
    for _, _, og, lg, out, lse, _ in cases:
        assert torch.equal(og, out) and torch.equal(lg, lse)


def test_attn_lengths_may_change_under_a_graph():
    c = Cache([400, 90], 16, 576, seed=22)
    cache, table, lens = c.to_gpu()
    q = torch.randn(2, 32, 576, generator=gen(23)).to(torch.bfloat16)
    qd = q.to(DEV)
    out, lse = torch.empty(2, 32, 512, dtype=torch.bfloat16, device=DEV), torch.empty(2, 32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_latent_attn(qd, cache, table, lens, out=out, lse=lse, scale=0.07)
    for now in ([400, 90], [1, 0], [129, 17], [400, 1]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_attn(out, lse, oracle(q, [k[:n] for k, n in zip(c.keys, now)], [1, 1], 512, 0.07))


@pytest.mark.parametrize("seed", range(24))
def test_attn_random_shapes_match(seed):
    g = gen(500 + seed)
    pick = lambda *v: v[int(torch.randint(0, len(v), (1,), generator=g))]
    N, H, page = pick(1, 2, 5), pick(1, 4, 12, 20, 32, 40, 64, 96), pick(16, 32, 64, 128)
    dv, dr = pick((512, 64), (512, 64), (512, 0), (256, 64), (256, 0))
    counts = torch.randint(0, pick(2, 4, 20) + 1, (N,), generator=g).tolist()
    counts[0] = max(1, counts[0])
    lens = torch.randint(0, pick(3, 70, 600, 1500), (N,), generator=g).tolist()
    causal = pick(True, True, False)
    c = Cache(lens, page, dv + dr, seed=seed, poison=pick(float("nan"), 1e30), gap=pick(0, 8, 64 * 576))
    q, out, lse, scale = run_attn(c, counts, H, dv, seed=seed, causal=causal, varlen=True, qscale=pick(1.0, 1.0, 8.0))
    assert kda.kda_get_device_error() == 0
    check_attn(out, lse, oracle(q, c.keys, counts, dv, scale, causal))


def test_attn_many_short_sequences():
    """More sequences than threads, some without tokens, some without keys."""
    g = gen(41)
    N = 1500
    lens = torch.randint(0, 4, (N,), generator=g).tolist()
    counts = torch.randint(0, 3, (N,), generator=g).tolist()
    c = Cache(lens, 16, 576, seed=41)
    q, out, lse, scale = run_attn(c, counts, 2, 512)
    assert kda.kda_get_device_error() == 0
    check_attn(out, lse, oracle(q, c.keys, counts, 512, scale))


def test_attn_long_sequence_in_many_pieces():
    """One sequence over every SM, and a bad page in the middle of it: nothing
    of the split tile is written."""
    n = 70000
    keys = torch.randn(n, 576, generator=gen(42)).to(torch.bfloat16)
    pages = -(-n // 16)
    cache = torch.zeros(pages * 16, 576, dtype=torch.bfloat16)
    cache[:n] = keys
    order = torch.randperm(pages, generator=gen(43))
    shuffled = torch.empty_like(cache).view(pages, 16, 576)
    shuffled[order] = cache.view(pages, 16, 576)
    dev, table = shuffled.to(DEV), order.int()[None].to(DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    q = torch.randn(2, 8, 576, generator=gen(44)).to(torch.bfloat16)
    out, lse = kda.kda_latent_attn(q.to(DEV), dev, table, lens, scale=0.07)
    assert kda.kda_get_device_error() == 0
    check_attn(out, lse, oracle(q, [keys], [2], 512, 0.07))
    table[0, 2500] = -3
    out.fill_(7)
    lse.fill_(7)
    kda.kda_latent_attn(q.to(DEV), dev, table, lens, out=out, lse=lse, scale=0.07)
    assert kda.kda_get_device_error() == 5
    assert (out == 7).all() and (lse == 7).all()


def test_attn_two_streams_at_once():
    cases = []
    for seed, lens, counts in ((51, [4000, 300], [1, 1]), (52, [900, 2500], [6, 6])):
        c = Cache(lens, 64, 576, seed=seed)
        q, out, lse, scale = run_attn(c, counts, 32, 512, seed=seed)
        cases.append((torch.cuda.Stream(), q.to(DEV), *c.to_gpu(), scale, out, lse, []))
    torch.cuda.synchronize()
    for _ in range(30):
        for stream, q, cache, table, lens, scale, _, _, got in cases:
            with torch.cuda.stream(stream):
                got.append(kda.kda_latent_attn(q, cache, table, lens, scale=scale))
    torch.cuda.synchronize()
    assert kda.kda_get_device_error() == 0
    for *_, out, lse, got in cases:
        assert all(torch.equal(o, out) and torch.equal(s, lse) for o, s in got)


# ------------------------------------------------------------------ rotary positions
def rotate64(x, pos, freqs, interleaved, inverse=False, scale=1.0):
    """x [T,H,rot] in 64 bits."""
    x = x.double()
    a = pos.double()[:, None] * freqs.double()[None, :] * (-1 if inverse else 1)
    c, s = a.cos()[:, None], a.sin()[:, None]
    h = x.shape[-1] // 2
    u, v = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    y = torch.empty_like(x)
    yu, yv = scale * (u * c - v * s), scale * (u * s + v * c)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = yu, yv
    else:
        y[..., :h], y[..., h:] = yu, yv
    return y


def check_rotated(y, x, ref, interleaved, scale):
    h = x.shape[-1] // 2
    xd = x.double()
    u, v = (xd[..., 0::2], xd[..., 1::2]) if interleaved else (xd[..., :h], xd[..., h:])
    size = abs(scale) * torch.hypot(u, v)
    size = torch.stack([size, size], -1).flatten(-2) if interleaved else torch.cat([size, size], -1)
    half = torch.finfo(y.dtype).eps / 2
    tol = half * ref.abs() + 2.0 ** -20 * size * (1 + half)
    bad = (y.double().cpu() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} off, worst {float(((y.double().cpu() - ref).abs() / tol.clamp_min(1e-300)).max())}"


def freqs_of(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,d,rot,offset", [(1, 1, 64, 64, 0), (3, 2, 128, 64, 64), (257, 5, 192, 64, 128),
                                              (5, 33, 96, 16, 80), (70, 1, 576, 64, 512), (9, 3, 128, 128, 0),
                                              (2, 1, 1024, 1024, 0), (4, 2, 72, 16, 8), (6, 1, 16, 16, 0)])
def test_rope_matches_the_formula(T, H, d, rot, offset, interleaved, dtype):
    x = torch.randn(T, H, d, generator=gen(T + d)).to(dtype)
    pos = torch.randint(-5, 1 << 21, (T,), generator=gen(T), dtype=torch.int32)
    pos[0] = 2 ** 31 - 1 if T > 1 else 12345
    f = freqs_of(rot)
    for inverse, scale in ((False, 1.0), (True, 1.25)):
        y = kda.kda_rope(x.to(DEV), pos.to(DEV), f.to(DEV), offset=offset, interleaved=interleaved, inverse=inverse, scale=scale)
        part = x[..., offset:offset + rot]
        ref = rotate64(part, pos, f, interleaved, inverse, scale)
        check_rotated(y[..., offset:offset + rot], part, ref, interleaved, scale)
        keep = torch.ones(d, dtype=torch.bool)
        keep[offset:offset + rot] = False
        assert torch.equal(y.cpu()[..., keep], x[..., keep])
        z = x.to(DEV)
        assert kda.kda_rope(z, pos.to(DEV), f.to(DEV), out=z, offset=offset, interleaved=interleaved, inverse=inverse,
                            scale=scale) is z
        assert torch.equal(z, y)


def test_rope_strided_tokens_both_ways():
    T, H, d = 37, 4, 64
    wide = torch.randn(T, 3 * H * d, generator=gen(2)).to(torch.bfloat16).to(DEV)
    x = wide[:, H * d:2 * H * d].view(T, H, d)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    f = freqs_of(32).to(DEV)
    y = kda.kda_rope(x.contiguous(), pos, f, offset=16)
    before = wide.clone()
    out = torch.zeros(T, 2 * H * d, dtype=torch.bfloat16, device=DEV)
    got = kda.kda_rope(x, pos, f, out=out[:, :H * d].view(T, H, d), offset=16)
    assert torch.equal(got, y) and (out[:, H * d:] == 0).all() and torch.equal(wide, before)
    kda.kda_rope(x, pos, f, out=x, offset=16)                           # in place on the slice
    assert torch.equal(x, y)
    before[:, H * d:2 * H * d] = y.reshape(T, -1)
    assert torch.equal(wide, before)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """inverse is the transposed map: against autograd of the formula, and
    against differences (the map is linear)."""
    T, H, d, rot, off = 6, 2, 64, 32, 16
    x = torch.randn(T, H, d, generator=gen(31), dtype=torch.float64)
    dy = torch.randn(T, H, d, generator=gen(32))
    pos = torch.randint(0, 1 << 20, (T,), generator=gen(33), dtype=torch.int32)
    f = freqs_of(rot)
    x.requires_grad_(True)
    y = torch.cat([x[..., :off], rotate64(x[..., off:off + rot], pos, f, interleaved, scale=1.3), x[..., off + rot:]], -1)
    (y * dy.double()).sum().backward()
    dx = kda.kda_rope(dy.to(DEV), pos.to(DEV), f.to(DEV), offset=off, interleaved=interleaved, inverse=True, scale=1.3)
    check_rotated(dx[..., off:off + rot], dy[..., off:off + rot], x.grad[..., off:off + rot], interleaved, 1.3)
    e = torch.randn(T, H, d, generator=gen(34))
    fwd = lambda v: kda.kda_rope(v.to(DEV), pos.to(DEV), f.to(DEV), offset=off, interleaved=interleaved, scale=1.3).double()
    base = x.detach().float()
    step = fwd(base + e) - fwd(base - e)
    # 2^-24 of values up to about 10 in 768 terms, on either side
    assert abs(float((step.cpu() * dy.double()).sum() - 2 * (dx.double().cpu() * e.double()).sum())) < 2e-2 * 2 ** -6


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,lens,page,H,dk,rot,interleaved", [
    ([1], [1], 16, 1, 576, 64, True),
    ([1, 1, 1], [5, 64, 65], 64, 32, 576, 64, False),
    ([3, 0, 40], [3, 7, 100], 16, 5, 320, 64, True),
    ([20, 20], [20, 333], 32, 16, 576, 64, False),
    ([7], [300], 128, 2, 64, 64, True),
])
def test_append_matches_the_formula(counts, lens, page, H, dk, rot, interleaved, dtype):
    T, extra = sum(counts), 2
    c = Cache(lens, page, dk, seed=T, dtype=dtype)
    cache, table, ln = c.to_gpu()
    before = cache.clone()
    wide = torch.randn(T + extra, dk + 8, generator=gen(41)).to(dtype)
    kv = wide[:, :dk]
    q_src = torch.randn(T + extra, H, 128 + rot, generator=gen(42)).to(dtype)
    q_pe = q_src[..., 128:]
    q0 = torch.randn(T + extra, H, dk, generator=gen(43)).to(dtype)
    q = q0.to(DEV)
    f = freqs_of(rot)
    cu = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32, device=DEV)
    kda.kda_latent_append(wide.to(DEV)[:, :dk], cache, table, ln, q_pe=q_src.to(DEV)[..., 128:], q=q, freqs=f.to(DEV),
                          cu_seqlens=cu, interleaved=interleaved, scale=0.9)
    assert kda.kda_get_device_error() == 0
    t, expect = 0, before.cpu()
    got = cache.cpu()
    for n, count in enumerate(counts):
        for i in range(count):
            p = lens[n] - count + i
            pg, r = int(c.table[n, p // page]), p % page
            pos = torch.tensor([p])
            row = got[pg, r].clone()
            assert torch.equal(row[:dk - rot], kv[t, :dk - rot])
            part = kv[t, dk - rot:][None, None]
            check_rotated(row[dk - rot:][None, None], part, rotate64(part, pos, f, interleaved, scale=0.9), interleaved, 0.9)
            check_rotated(q[t:t + 1, :, dk - rot:], q_pe[t:t + 1], rotate64(q_pe[t:t + 1], pos, f, interleaved, scale=0.9),
                          interleaved, 0.9)
            expect[pg, r] = row
            t += 1
    assert torch.equal(torch.nan_to_num(got.float(), 123.0), torch.nan_to_num(expect.float(), 123.0))
    assert torch.equal(q.cpu()[..., :dk - rot], q0[..., :dk - rot])
    assert torch.equal(q.cpu()[T:], q0[T:])                    # rows behind the last sequence


def test_append_without_positions():
    c = Cache([40, 9], 16, 576, seed=51)
    cache, table, lens = c.to_gpu()
    kv = torch.randn(4, 576, generator=gen(52)).to(torch.bfloat16).to(DEV)
    q_pe = torch.randn(4, 3, 64, generator=gen(53)).to(torch.bfloat16).to(DEV)
    q = torch.zeros(4, 3, 576, dtype=torch.bfloat16, device=DEV)
    kda.kda_latent_append(kv, cache, table, lens, q_pe=q_pe, q=q)
    assert torch.equal(q[..., 512:], q_pe) and (q[..., :512] == 0).all()
    for t, (n, p) in enumerate([(0, 38), (0, 39), (1, 7), (1, 8)]):
        assert torch.equal(cache[int(c.table[n, p // 16]), p % 16], kv[t])


def test_append_skips_and_reports_bad_places():
    c = Cache([20, 3, 40], 16, 576, seed=54)
    c.table[0, 1] = c.cache.shape[0]        # positions 16..19 of the first sequence
    cache, table, lens = c.to_gpu()
    before = cache.clone()
    kv = torch.randn(15, 576, generator=gen(55)).to(torch.bfloat16).to(DEV)     # 5 each: two of the second sequence before 0
    kda.kda_latent_append(kv, cache, table, lens)
    assert kda.kda_get_device_error() == 5
    before[int(c.table[0, 0]), 15] = kv[0]
    for t, p in ((7, 0), (8, 1), (9, 2)):
        before[int(c.table[1, 0]), p] = kv[t]
    for t in range(5):
        p = 35 + t
        before[int(c.table[2, p // 16]), p % 16] = kv[10 + t]
    assert torch.equal(torch.nan_to_num(cache.float(), 123.0), torch.nan_to_num(before.float(), 123.0))


def test_sequences_are_found_among_many():
    """The search over the offsets: 3000 sequences of 0 to 3 tokens."""
    counts = torch.randint(0, 4, (3000,), generator=gen(56)).tolist()
    N, T = len(counts), sum(counts)
    table = torch.arange(N, dtype=torch.int32, device=DEV).view(N, 1)
    lens = torch.tensor(counts, dtype=torch.int32, device=DEV)
    cache = torch.zeros(N, 16, 64, device=DEV)
    kv = torch.randn(T, 64, generator=gen(57)).to(DEV)
    cu = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32, device=DEV)
    kda.kda_latent_append(kv, cache, table, lens, cu_seqlens=cu)
    seq = torch.repeat_interleave(torch.arange(N), torch.tensor(counts))
    at = torch.cat([torch.arange(c) for c in counts])
    expect = torch.zeros_like(cache)
    expect[seq.to(DEV), at.to(DEV)] = kv
    assert kda.kda_get_device_error() == 0
    assert torch.equal(cache, expect)


# ------------------------------------------------------------------ pages
def plain_copy(pool, src, dst):
    """[planes, pages, ...]; in order, from a copy."""
    old = pool.clone()
    for s, d in zip(src, dst):
        pool[:, d] = old[:, s] if s >= 0 else 0
    return pool


@pytest.mark.parametrize("shape,planes,moves", [
    ((5, 4), False, [(0, 3)]),
    ((7, 3, 12), False, [(1, 2), (2, 1)]),                                  # exchange
    ((9, 40), False, [(0, 1), (1, 2), (2, 3), (3, 0), (4, 4)]),              # rotation, one onto itself
    ((3, 8, 100), True, [(0, 7), (0, 6), (0, 5), (-1, 0)]),                  # fork, then clear the source
    ((1, 4, 8), True, [(0, 1), (2, 1), (3, 1)]),                            # the last move counts
    ((2, 6, 1000), True, [(5, 5), (1, 0), (1, 0), (-1, 3), (4, 3)]),
    ((4, 32 * 1024), False, [(3, 0), (0, 3), (1, 2)]),
])
def test_copy_matches_moves_in_order(shape, planes, moves):
    pool = torch.randn(*shape, generator=gen(61))
    src, dst = [m[0] for m in moves], [m[1] for m in moves]
    dev = pool.to(DEV)
    kda.kda_pages_copy(dev, torch.tensor(src, dtype=torch.int32, device=DEV), torch.tensor(dst, dtype=torch.int32, device=DEV),
                       planes=planes)
    assert kda.kda_get_device_error() == 0
    assert torch.equal(dev.cpu(), plain_copy(pool if planes else pool[None], src, dst).view(shape))


@pytest.mark.parametrize("pages,words,count", [(300, 4, 299), (5000, 4, 4096), (5000, 12, 4096), (1000, 516, 700), (64, 20000, 64),
                                               (3, 4, 4096)])
def test_copy_many_random_moves(pages, words, count):
    pool = torch.randn(pages, words, generator=gen(62))
    src = torch.randint(-1, pages, (count,), generator=gen(63), dtype=torch.int32)
    dst = torch.randint(0, pages, (count,), generator=gen(64), dtype=torch.int32)
    dev = pool.to(DEV)
    kda.kda_pages_copy(dev, src.to(DEV), dst.to(DEV))
    old = pool.clone()
    for s, d in zip(src.tolist(), dst.tolist()):
        pool[d] = old[s] if s >= 0 else 0
    assert torch.equal(dev.cpu(), pool)


def test_copy_skips_and_reports_bad_pages():
    pool = torch.randn(6, 64, generator=gen(65))
    src = [0, 6, 2, -2, 1, 3]
    dst = [5, 4, 6, 3, -1, 4]
    dev = pool.to(DEV)
    kda.kda_pages_copy(dev, torch.tensor(src, dtype=torch.int32, device=DEV), torch.tensor(dst, dtype=torch.int32, device=DEV))
    assert kda.kda_get_device_error() == 3
    assert torch.equal(dev.cpu(), plain_copy(pool[None], [0, 3], [5, 4])[0])


def test_moves_past_32_bits():
    """A pool of 6 GB: pages beyond 2^32 bytes, copied and compacted."""
    pages, words = 3000, 1 << 19
    pool = torch.zeros(pages, words, device=DEV)
    for i in (5, 2200, 2999):
        pool[i] = torch.arange(words, device=DEV, dtype=torch.float32) + i
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    kda.kda_pages_copy(pool, t(2999, 5), t(2500, 2999))
    ramp = torch.arange(words, device=DEV, dtype=torch.float32)
    assert torch.equal(pool[2500], ramp + 2999) and torch.equal(pool[2999], ramp + 5)
    new = kda.kda_pages_compact(pool, t(2500, 2200, 2999))
    assert new.tolist() == [1, 0, 2]
    assert torch.equal(pool[0], ramp + 2200) and torch.equal(pool[1], ramp + 2999) and torch.equal(pool[2], ramp + 5)


def plain_compact(pages, n_pages):
    live = sorted({p for p in pages if 0 <= p < n_pages})
    n = len(live)
    holes = [i for i in range(n) if i not in set(live)]
    name = dict(zip([p for p in live if p >= n], holes))
    return name, [name.get(p, p) for p in pages]


@pytest.mark.parametrize("n_pages,live,extra,planes,words", [
    (1, 1, 0, 1, 4), (8, 8, 3, 1, 4), (8, 1, 0, 2, 36), (40, 17, 9, 3, 260), (1000, 333, 100, 1, 5000),
    (70000, 30000, 5000, 1, 4), (33, 32, 0, 1, 20000), (524288, 100, 7, 1, 4)])
def test_compact_matches_the_rule(n_pages, live, extra, planes, words):
    g = gen(n_pages + live)
    perm = torch.randperm(n_pages, generator=g)[:live]
    listed = torch.cat([perm, perm[:extra], torch.full((extra,), -1), torch.full((1 if extra else 0,), -7)])
    listed = listed[torch.randperm(len(listed), generator=g)].int()
    pool = torch.randn(planes, n_pages, words, generator=g)
    dev = pool.to(DEV)
    got = kda.kda_pages_compact(dev, listed.to(DEV), planes=True)
    assert kda.kda_get_device_error() == 0
    name, new = plain_compact(listed.tolist(), n_pages)
    assert got.tolist() == new
    keep = listed >= 0
    assert torch.equal(dev.cpu()[:, torch.tensor(new)[keep].long()], pool[:, listed[keep].long()])


def test_compact_in_place_on_a_table_and_bad_entries():
    pool = torch.arange(10, dtype=torch.float32)[:, None].repeat(1, 8).to(DEV)
    table = torch.tensor([[9, -1, 3], [3, 12, 0]], dtype=torch.int32, device=DEV)
    assert kda.kda_pages_compact(pool, table, out=table) is table
    assert kda.kda_get_device_error() == 3
    assert table.tolist() == [[2, -1, 1], [1, 12, 0]]
    assert pool[:3, 0].tolist() == [0, 3, 9]


def test_compact_only_padding_moves_nothing():
    pool = torch.randn(6, 8, generator=gen(71)).to(DEV)
    before = pool.clone()
    new = kda.kda_pages_compact(pool, torch.full((5,), -1, dtype=torch.int32, device=DEV))
    assert torch.equal(pool, before) and (new == -1).all()


# ------------------------------------------------------------------ together
def test_a_serving_run_of_a_hybrid():
    """A KDA layer on its slot pool and a latent layer on its paged cache: a
    prompt chunk, decode steps, a fork (state copied, the last page copied, the
    full ones shared), more steps, then both pools compacted: every
    sequence's outputs match those of its own uninterrupted run."""
    H, d, page, dk = 4, 128, 16, 576
    f = freqs_of(64).to(DEV)
    tok = lambda s, n: torch.randn(n, dk, generator=gen(s)).to(torch.bfloat16).to(DEV)
    qry = lambda s, n: torch.randn(n, H, dk, generator=gen(1000 + s)).to(torch.bfloat16).to(DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)

    def latent(cache, table, lens, kv, q, cu):
        q = q.clone()
        kda.kda_latent_append(kv, cache, table, lens, q_pe=q[..., 512:].contiguous(), q=q, freqs=f, cu_seqlens=cu)
        return kda.kda_latent_attn(q, cache, table, lens, cu_seqlens=cu, scale=0.07)[0]

    def delta(pool, slots, seeds):
        x = [W.decode_tokens(s, 1, H, d, d, seed=7) for s in seeds]
        x = [torch.stack([t[i] for t in x], 1)[0][:, None].contiguous().to(DEV) for i in range(5)]
        return kda.kda_recurrent_steps(*x, pool, slots)

    cache = torch.full((12, page, dk), float("nan"), dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(6, H, d, d, device=DEV)
    table = torch.full((3, 4), -1, dtype=torch.int32, device=DEV)
    table[0, :2], table[1, :2] = i32(11, 7), i32(2, 9)
    # two sequences: prompts of 20 and 3 tokens, then a token each
    latent(cache, table[:2].contiguous(), i32(20, 3), torch.cat([tok(1, 20), tok(2, 3)]), torch.cat([qry(1, 20), qry(2, 3)]), i32(0, 20, 23))
    s1 = delta(pool, i32(5, 1), [10, 20])
    latent(cache, table[:2].contiguous(), i32(21, 4), torch.cat([tok(3, 1), tok(4, 1)]), torch.cat([qry(3, 1), qry(4, 1)]), None)
    # the first one forks: state slot 5 -> 3; page 11 is full and shared, page 7 is copied to 4
    kda.kda_pages_copy(pool, i32(5), i32(3))
    kda.kda_pages_copy(cache, i32(7), i32(4))
    table[2, :2] = i32(11, 4)
    o1 = latent(cache, table, i32(22, 5, 22), torch.cat([tok(5, 1), tok(6, 1), tok(7, 1)]), torch.cat([qry(5, 1), qry(6, 1), qry(7, 1)]), None)
    s2 = delta(pool, i32(5, 1, 3), [11, 21, 31])
    # the second one ends; what is left moves to the front
    slots = kda.kda_pages_compact(pool, i32(5, 3))
    left = table[[0, 2]].contiguous()
    kda.kda_pages_compact(cache, left, out=left)
    assert sorted(set(left.flatten().tolist())) == [-1, 0, 1, 2] and sorted(slots.tolist()) == [0, 1]
    o2 = latent(cache, left, i32(23, 23), torch.cat([tok(8, 1), tok(9, 1)]), torch.cat([qry(8, 1), qry(9, 1)]), None)
    s3 = delta(pool, slots, [12, 32])
    assert kda.kda_get_device_error() == 0

    def alone(kv, q, page_ids, at, n):
        """The last n tokens' attention in a cache of its own, one chunk."""
        c = torch.full((12, page, dk), float("nan"), dtype=torch.bfloat16, device=DEV)
        return latent(c, i32(*page_ids)[None], i32(at), kv, q, i32(0, at))[-n:]

    parent = [(1, 20), (3, 1), (5, 1), (8, 1)]
    child = [(1, 20), (3, 1), (7, 1), (9, 1)]
    for k, path in enumerate((parent, child)):
        ref = alone(torch.cat([tok(s, n) for s, n in path]), torch.cat([qry(s, n) for s, n in path]), [0, 1], 23, 2)
        mine = torch.stack([o1[0 if k == 0 else 2], o2[k]])
        # both are rounded to bf16, with probabilities that were, in another split: values of order 1 in
        # 22 or 23 weights, each side off by U (|out| + A) with A < 3
        assert float((ref.float() - mine.float()).abs().max()) < 2 * U * (ref.float().abs().max() + 3)
    for k, seeds in enumerate(([10, 11, 12], [10, 31, 32])):
        own = torch.zeros(1, H, d, d, device=DEV)
        ref = torch.cat([delta(own, i32(0), [s]) for s in seeds])
        assert torch.equal(ref[1], s2[0 if k == 0 else 2]) and torch.equal(ref[2], s3[k])


def _refused_calls():
    """name -> (exception, call on a dict of good arguments): what the binding or the library turns away on the host."""
    V, Ty, K = ValueError, TypeError, kda.KDAError
    return {
        "attn q of two dimensions": (V, lambda a: kda.kda_latent_attn(a["q"][0], a["cache"], a["table"], a["lens"])),
        "attn q strided": (V, lambda a: kda.kda_latent_attn(a["q"][:, ::2], a["cache"], a["table"], a["lens"])),
        "attn q fp16": (Ty, lambda a: kda.kda_latent_attn(a["q"].half(), a["cache"], a["table"], a["lens"])),
        "attn all fp16": (K, lambda a: kda.kda_latent_attn(a["q"].half(), a["cache"].half(), a["table"], a["lens"])),
        "attn all fp32": (K, lambda a: kda.kda_latent_attn(a["q"].float(), a["cache"].float(), a["table"], a["lens"])),
        "attn cache on the host": (Ty, lambda a: kda.kda_latent_attn(a["q"], a["cache"].cpu(), a["table"], a["lens"])),
        "attn cache of other rows": (V, lambda a: kda.kda_latent_attn(a["q"], a["cache"][..., :512], a["table"], a["lens"])),
        "attn page rows apart": (V, lambda a: kda.kda_latent_attn(a["q"], a["cache"][:, ::2], a["table"], a["lens"])),
        "attn table of 64 bits": (Ty, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"].long(), a["lens"])),
        "attn table strided": (V, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"][:, ::2], a["lens"])),
        "attn table of other rows": (V, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"][:1], a["lens"])),
        "attn lens on the host": (V, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"].cpu())),
        "attn no lens": (Ty, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], None)),
        "attn offsets of other length": (V, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"], cu_seqlens=a["lens"])),
        "attn tokens that do not divide": (V, lambda a: kda.kda_latent_attn(a["q"][:1], a["cache"], a["table"], a["lens"])),
        "attn out of other shape": (V, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"], out=a["q"])),
        "attn out of other type": (Ty, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"],
                                                                     out=a["q"][..., :512].float().contiguous())),
        "attn lse bf16": (Ty, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"],
                                                            lse=a["q"][..., 0].contiguous())),
        "attn scale inf": (K, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"], scale=float("inf"))),
        "attn dv negative": (V, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"], dv=-1)),
        "attn dv 0": (K, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"], dv=0)),
        "attn dv past 32 bits": (V, lambda a: kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"], dv=1 << 33)),
        "append rows apart": (V, lambda a: kda.kda_latent_append(a["wide"][:, ::2], a["cache"], a["table"], a["lens"])),
        "append broadcast rows": (V, lambda a: kda.kda_latent_append(a["kv"][:1].expand(2, 576), a["cache"], a["table"], a["lens"])),
        "append q_pe alone": (V, lambda a: kda.kda_latent_append(a["kv"], a["cache"], a["table"], a["lens"], q_pe=a["q_pe"], freqs=a["freqs"])),
        "append q alone": (V, lambda a: kda.kda_latent_append(a["kv"], a["cache"], a["table"], a["lens"], q=a["q"], freqs=a["freqs"])),
        "append q_pe of other width": (V, lambda a: kda.kda_latent_append(a["kv"], a["cache"], a["table"], a["lens"], q_pe=a["q_pe"][..., :62],
                                                                          q=a["q"], freqs=a["freqs"])),
        "append q_pe broadcast": (V, lambda a: kda.kda_latent_append(a["kv"], a["cache"], a["table"], a["lens"], q_pe=a["q_pe"][:, :1].expand(2, 4, 64),
                                                                     q=a["q"], freqs=a["freqs"])),
        "append q of other heads": (V, lambda a: kda.kda_latent_append(a["kv"], a["cache"], a["table"], a["lens"], q_pe=a["q_pe"][:, :3],
                                                                       q=a["q"], freqs=a["freqs"])),
        "append freqs bf16": (Ty, lambda a: kda.kda_latent_append(a["kv"], a["cache"], a["table"], a["lens"], freqs=a["freqs"].bfloat16())),
        "rope heads apart": (V, lambda a: kda.kda_rope(a["q"][:, ::2], a["lens"], a["freqs"])),
        "rope positions of 64 bits": (Ty, lambda a: kda.kda_rope(a["q"], a["lens"].long(), a["freqs"])),
        "rope positions of other length": (V, lambda a: kda.kda_rope(a["q"], a["lens"][:1], a["freqs"])),
        "rope beyond the head": (K, lambda a: kda.kda_rope(a["q"], a["lens"], a["freqs"], offset=576)),
        "rope offset past 32 bits": (V, lambda a: kda.kda_rope(a["q"], a["lens"], a["freqs"], offset=1 << 32)),
        "rope out of other type": (V, lambda a: kda.kda_rope(a["q"], a["lens"], a["freqs"], out=a["q"].float())),
        "rope out broadcast": (V, lambda a: kda.kda_rope(a["q"], a["lens"], a["freqs"], out=a["q"][:1].expand(2, 4, 576))),
        "rope fp16": (K, lambda a: kda.kda_rope(a["q"].half(), a["lens"], a["freqs"])),
        "copy pool strided": (V, lambda a: kda.kda_pages_copy(a["cache"][:, ::2], a["lens"], a["lens"])),
        "copy lists of two lengths": (V, lambda a: kda.kda_pages_copy(a["cache"], a["lens"], a["lens"][:1])),
        "copy lists of 64 bits": (Ty, lambda a: kda.kda_pages_copy(a["cache"], a["lens"].long(), a["lens"].long())),
        "copy planes of a flat pool": (V, lambda a: kda.kda_pages_copy(a["cache"][0], a["lens"], a["lens"], planes=True)),
        "copy empty pool": (V, lambda a: kda.kda_pages_copy(a["cache"][:0], a["lens"], a["lens"])),
        "compact out of other shape": (V, lambda a: kda.kda_pages_compact(a["cache"], a["table"], out=a["lens"])),
        "compact pages on the host": (V, lambda a: kda.kda_pages_compact(a["cache"], a["table"].cpu())),
    }


def _good_arguments():
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    return dict(q=torch.ones(2, 4, 576, **bf), cache=torch.ones(6, 32, 576, **bf), kv=torch.ones(2, 576, **bf),
                wide=torch.ones(2, 1152, **bf), q_pe=torch.ones(2, 4, 64, **bf), freqs=torch.ones(32, device="cuda"),
                table=torch.arange(6, **i32).view(2, 3), lens=torch.tensor([3, 4], **i32))


@pytest.mark.parametrize("what", list(_refused_calls()))
def test_refused_calls_leave_everything_as_it_was(what):
    error, call = _refused_calls()[what]
    a = _good_arguments()
    before = {k: v.clone() for k, v in a.items()}
    with pytest.raises(error) as got:
        call(a)
    if error is kda.KDAError:
        assert got.value.status in (1, 2) and "kda_" in str(got.value)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], before[k]) for k in a)
    assert kda.kda_get_device_error() == 0
    out, _ = kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"])      # the next call is not affected
    assert torch.equal(out, torch.ones_like(out))


def test_default_scale_and_accepted_forms():
    a = _good_arguments()
    gen = torch.Generator(device="cuda").manual_seed(3)
    a["q"].normal_(generator=gen)
    a["cache"].normal_(generator=gen)
    want = kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"], scale=576 ** -0.5)
    got = kda.kda_latent_attn(q=a["q"], cache=a["cache"], page_table=a["table"], kv_lens=a["lens"], causal=1)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    whole = kda.kda_latent_attn(a["q"], a["cache"], a["table"], a["lens"], scale=1)
    assert torch.isfinite(whole[0]).all()
    none = kda.kda_latent_attn(a["q"][:0], a["cache"], a["table"], a["lens"])
    assert none[0].shape == (0, 4, 512) and none[1].shape == (0, 4)
    out = torch.empty_like(a["q"])
    assert kda.kda_rope(a["q"], a["lens"], a["freqs"], out=out) is not None
    assert torch.equal(out, kda.kda_rope(a["q"], a["lens"], a["freqs"]))


def test_two_threads_call_at_once():
    args = []
    for seed in range(2):
        a = _good_arguments()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        a["q"].normal_(generator=gen)
        a["cache"].normal_(generator=gen)
        args.append(a)

    def one(a):
        x = kda.kda_rope(a["q"], a["lens"], a["freqs"], offset=512)
        return kda.kda_latent_attn(x, a["cache"], a["table"], a["lens"])

    want = [one(a) for a in args]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    got = one(args[i])
                    if not (torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])):
                        bad.append(i)
                    try:
                        kda.kda_rope(args[i]["q"], args[i]["lens"], args[i]["freqs"], offset=576 + i)
                        bad.append("accepted")
                    except kda.KDAError as e:            # each thread has its own message
                        if f"offset={576 + i}" not in str(e):
                            bad.append(str(e))
        except Exception as e:
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]
