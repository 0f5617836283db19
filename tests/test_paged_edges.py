"""Edges of the paged latent cache's operators: calls at the ends of what the
header allows, against plain 64-bit forms and exact integer arithmetic (B200).

The bounds of the attention's errors are those of test_paged_latent.py; others
stand beside their tests.
"""
import math
import threading
from fractions import Fraction

import pytest
import torch

import gated_delta_rule_88_b200 as kda
from test_paged_latent import DEV, Cache, check_attn, check_rotated, freqs_of, gen, oracle, rotate64, run_attn

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ refused on the host
@pytest.mark.parametrize("how", ["attention", "append"])
def test_cache_of_one_page_repeated_is_refused(how):
    """expand() gives pages a stride of 0, which the library would take for its default."""
    cache = torch.ones(1, 32, 576, dtype=torch.bfloat16, device=DEV).expand(6, 32, 576)
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    lens = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    x = torch.ones(2, 4, 576, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        if how == "attention":
            kda.kda_latent_attn(x, cache, table, lens)
        else:
            kda.kda_latent_append(x[:, 0], cache, table, lens)
    # one page of any stride is a pool of one page
    out, _ = kda.kda_latent_attn(x, cache[:1], torch.zeros_like(table), lens)
    assert kda.kda_get_device_error() == 0 and torch.equal(out, torch.ones_like(out))


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("page", [16, 128])
def test_attn_longest_sequence(page):
    """2^31 - 256 keys, all of them in one page that the whole table names: the
    answer is that page's.  Sums of 2^31 / 148 equal shares, a tile of 64 after
    the other, in fp32: a thread's sum takes n / (148 64) additions of half a unit in
    the last place at most (2^-24), the accumulators four products each, truncated
    (2^-23); both relative to the sum of the absolute terms."""
    n, dk, H = 2 ** 31 - 256, 256, 2
    keys = torch.randn(page, dk, generator=gen(page)).to(torch.bfloat16)
    q = torch.randn(1, H, dk, generator=gen(1)).to(torch.bfloat16)
    table = torch.ones(1, n // page, dtype=torch.int32, device=DEV)
    cache = torch.stack([torch.full_like(keys, float("nan")), keys]).to(DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    out, lse = kda.kda_latent_attn(q.to(DEV), cache, table, lens, dv=dk, scale=0.05)
    assert kda.kda_get_device_error() == 0
    x = torch.einsum("hd,kd->hk", q[0].double(), keys.double()) * 0.05
    p = torch.softmax(x, -1)
    tiles = n / (148 * 64)
    size = p @ keys.double().abs()
    sums = tiles * 2.0 ** -24
    assert float((lse[0].double().cpu() - torch.logsumexp(x, -1) - math.log(n // page)).abs().max()) < 1.1 * sums + 1e-4
    assert float(((out[0].double().cpu() - p @ keys.double()).abs() / size).max()) < 4 * tiles * 2.0 ** -23 + sums + 2.0 ** -7


# ------------------------------------------------------------------ lists of any length from two threads
def both_at_once(works):
    """Runs the functions in threads, 300 times each; the first exceptions or answers other than None."""
    bad, start = [], threading.Barrier(len(works))

    def loop(work):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(300):
                    got = work()
                    if got is not None:
                        bad.append(got)
        except Exception as e:
            bad.append(repr(e))

    threads = [threading.Thread(target=loop, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad[:3]


def test_two_threads_copy_long_and_short_lists():
    """The shared memory of a call (224 KB, a few KB) is no other call's limit."""
    works, pools = [], []
    for count in (4096, 3):
        pool = torch.randn(5000, 4, generator=gen(count)).to(DEV)
        src = torch.randperm(5000, generator=gen(count + 1))[:count].int().to(DEV)
        pools.append((pool, pool.clone()))
        works.append(lambda pool=pool, src=src: kda.kda_pages_copy(pool, src, src))          # each page onto itself
    assert not both_at_once(works)
    assert kda.kda_get_device_error() == 0
    assert all(torch.equal(a, b) for a, b in pools)


def test_two_threads_compact_large_and_small_pools():
    works, checks = [], []
    for n in (524288, 8):
        pool = torch.randn(n, 4, generator=gen(n)).to(DEV)
        live = torch.arange(3, dtype=torch.int32, device=DEV)                                 # in front already: nothing moves
        out = torch.empty_like(live)
        checks.append((pool, pool.clone(), out, live))
        works.append(lambda pool=pool, live=live, out=out: (kda.kda_pages_compact(pool, live, out=out), None)[1])
    assert not both_at_once(works)
    assert kda.kda_get_device_error() == 0
    assert all(torch.equal(a, b) and torch.equal(o, l) for a, b, o, l in checks)


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("lens,count,H", [([40], 1, 32), ([40, 250], 1, 128), ([100, 130], 2, 32), ([6000, 9000], 1, 8),
                                          ([6000], 4, 32)])
def test_attn_waits_that_run_out(lens, count, H):
    """The way out of a block with its copies under way (all of a short tile's, or
    a long range's first ones): the error word is set, nothing is written, and
    the next call is right."""
    c = Cache(lens, 64, 576, seed=60)
    cache, table, ln = c.to_gpu()
    N, T = len(lens), len(lens) * count
    q = torch.randn(T, H, 576, generator=gen(61)).to(torch.bfloat16)
    qd = q.to(DEV)
    out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H), 7.0, device=DEV)
    kda.kda_selftest_latent_attn(qd, cache, table, ln, out=out, lse=lse, scale=0.07)
    assert kda.kda_get_device_error() == 1
    assert (out == 7).all() and (lse == 7).all()
    kda.kda_latent_attn(qd, cache, table, ln, out=out, lse=lse, scale=0.07)
    assert kda.kda_get_device_error() == 0
    check_attn(out, lse, oracle(q, c.keys, [count] * N, 512, 0.07))


# ------------------------------------------------------------------ values and logits at the ends of their ranges
@pytest.mark.parametrize("n", [250, 300])
@pytest.mark.parametrize("rise", [15.5, 30.0, 59.0, 61.0, 200.0])
def test_attn_large_values_above_a_low_first_tile(n, rise):
    """Values of 2^100 whose logits rise by any amount after the first tile: the
    answer is finite and stays so on the way (kv_len times a value < 2^110)."""
    H, dk = 8, 576
    c = Cache([n], 64, dk, seed=n)
    k = torch.zeros(n, dk)
    k[:, :512] = torch.randn(n, 512, generator=gen(1)).clamp(-1, 1) * 2.0 ** 100
    k[64:, 512] = rise / 2                                   # powers of two above the first tile's logits
    k[128:, 512] = rise
    c.keys[0] = k.to(torch.bfloat16)
    for j in range(c.table.shape[1]):
        rows = c.keys[0][64 * j:64 * j + 64]
        c.cache[c.table[0, j], :len(rows)] = rows
    q = torch.zeros(1, H, dk, dtype=torch.bfloat16)
    q[..., 512] = 1
    cache, table, lens = c.to_gpu()
    out, lse = kda.kda_latent_attn(q.to(DEV), cache, table, lens, scale=math.log(2))
    assert kda.kda_get_device_error() == 0
    check_attn(out, lse, oracle(q, c.keys, [1], 512, math.log(2)))


@pytest.mark.parametrize("n", [250, 300])
@pytest.mark.parametrize("where", ["query", "key"])
def test_attn_nan_is_not_an_empty_row(where, n):
    """A NaN in a query, or in a key that a row sees, shows in its out and lse; -inf
    is the mark of a row that sees nothing."""
    H = 32
    c = Cache([n], 64, 576, seed=n)
    q = torch.randn(1, H, 576, generator=gen(2)).to(torch.bfloat16)
    if where == "query":
        q[0, 5, 17] = float("nan")
    cache, table, lens = c.to_gpu()
    if where == "key":
        cache[int(c.table[0, 1]), 6, 570] = float("nan")
    out, lse = kda.kda_latent_attn(q.to(DEV), cache, table, lens, scale=0.07)
    hit = torch.full((H,), where == "key")
    hit[5] = True
    assert lse[0, hit.to(DEV)].isnan().all() and out[0, hit.to(DEV)].isnan().all()
    if where == "query":
        q[0, 5] = 0
        ref = oracle(q, c.keys, [1], 512, 0.07)
        check_attn(out[:, ~hit.to(DEV)], lse[:, ~hit.to(DEV)], [x[:, ~hit] for x in ref])


# ------------------------------------------------------------------ angles
def two_pi(bits):
    """2 pi as an integer over 2^bits, by Machin's formula."""
    one = 1 << (bits + 16)

    def atan_inv(x):
        term, total, k = one // x, 0, 0
        while term:
            total += term // (2 * k + 1) * (-1) ** k
            term //= x * x
            k += 1
        return total

    return (8 * (4 * atan_inv(5) - atan_inv(239))) >> 16


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_angle_at_any_position(interleaved):
    """The angle is off by at most pi 2^-24 at any position and frequency: pairs
    (1, 0) give the cosine and the sine, each off by that and one unit in the last
    place of sincospif (2^-24 at most; the products with 1 and 0 are exact)."""
    pos = [2142271631, 2 ** 31 - 1, -2 ** 31, 1, 0, -7, 1 << 20]
    pos += torch.randint(-2 ** 31, 2 ** 31, (200,), generator=gen(3)).tolist()
    freqs = torch.tensor([1.0, 0.7498942, 0.031622775, 1e-6, 37.5, 1000.3, 3.0e5, 6.2831855], dtype=torch.float32)
    x = torch.zeros(len(pos), 1, 16)
    x[..., slice(0, None, 2) if interleaved else slice(0, 8)] = 1
    y = kda.kda_rope(x.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV), freqs.to(DEV), interleaved=interleaved)
    y = y.double().cpu()[:, 0]
    cos, sin = (y[:, 0::2], y[:, 1::2]) if interleaved else (y[:, :8], y[:, 8:])
    bits = 260
    turn = two_pi(bits)
    tol = math.pi * 2.0 ** -24 + 2.0 ** -24
    worst = 0.0
    for t, p in enumerate(pos):
        for i, f in enumerate(freqs.tolist()):
            a = int(Fraction(f) * p * (1 << bits)) % turn
            a = Fraction(a, 1 << bits)
            worst = max(worst, abs(math.cos(a) - float(cos[t, i])), abs(math.sin(a) - float(sin[t, i])))
    assert worst <= tol, f"{worst / tol:.2f} x the bound"


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("length", ["capacity + 1", "capacity + 5", "negative"])
def test_append_writes_nothing_of_a_sequence_of_impossible_length(length):
    c = Cache([20, 32, 40], 16, 576, seed=54)
    cap = c.table.shape[1] * 16
    for n in range(3):                                       # every entry is a page of its own
        c.table[n] = torch.arange(3) + 3 * n
    c.lens[1] = {"capacity + 1": cap + 1, "capacity + 5": cap + 5, "negative": -1}[length]
    table, lens = c.table.to(DEV), c.lens.to(DEV)
    cache = torch.full((9, 16, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    kv = torch.randn(15, 576, generator=gen(55)).to(torch.bfloat16).to(DEV)
    q_pe = torch.randn(15, 2, 64, generator=gen(56)).to(torch.bfloat16).to(DEV)
    q = torch.full((15, 2, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    kda.kda_latent_append(kv, cache, table, lens, q_pe=q_pe, q=q)
    assert kda.kda_get_device_error() == 5
    expect = torch.full_like(cache, 7.0)
    for t in range(5):
        expect[(15 + t) // 16, (15 + t) % 16] = kv[t]
        expect[6 + (35 + t) // 16, (35 + t) % 16] = kv[10 + t]
    assert torch.equal(cache, expect)
    assert torch.equal(q[:5, :, 512:], q_pe[:5]) and torch.equal(q[10:, :, 512:], q_pe[10:])
    assert (q[5:10] == 7).all() and (q[..., :512] == 7).all()


@pytest.mark.parametrize("T,H", [(3, 33), (2051, 4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("positions", ["halves", "interleaved", "none"])
def test_append_turns_the_queries_in_place(T, H, dtype, positions):
    """q_pe is the slice of q that is written: the bits of a call with a copy of it."""
    g = gen(T)
    kv, q = torch.randn(T, 128, generator=g).to(DEV, dtype), torch.randn(T, H, 128, generator=g).to(DEV, dtype)
    pages = -(-T // 16)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    freqs = None if positions == "none" else (10000.0 ** (-torch.arange(32) / 32.0)).to(DEV)
    made = []
    for copied in (True, False):
        mine, cache = q.clone(), torch.zeros(pages, 16, 128, dtype=dtype, device=DEV)
        part = mine[..., 64:].contiguous() if copied else mine[..., 64:]
        kda.kda_latent_append(kv, cache, table, lens, q_pe=part, q=mine, freqs=freqs, interleaved=positions == "interleaved")
        made.append((mine, cache))
    assert kda.kda_get_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(*made))
    assert torch.equal(made[0][0], q) == (positions == "none")


# ------------------------------------------------------------------ many row tiles, many tokens
def oracle_on_gpu(q, keys, counts, dv, scale):
    """oracle() of test_paged_latent.py for long causal chunks: whole sequences at once, on the GPU in 64 bits."""
    dk, H = q.shape[2], q.shape[1]
    parts, t = [], 0
    for k, count in zip(keys, counts):
        if not count:
            continue
        k, x = k.to(DEV).double(), q[t:t + count].to(DEV).double().reshape(-1, q.shape[2])
        see = len(k) - count + torch.arange(count, device=DEV).repeat_interleave(H) + 1
        hidden = torch.arange(len(k), device=DEV)[None] >= see[:, None]
        logits = (x @ k.T * scale).masked_fill_(hidden, -float("inf"))
        size = abs(scale) * (x.abs() @ k.abs().T).masked_fill_(hidden, 0).amax(-1)
        none = see <= 0
        p = torch.softmax(logits, -1).masked_fill_(none[:, None], 0)
        X = ((dk + 8) * 2.0 ** -24 * size + 2.0 ** -22)[:, None]
        A = p @ k[:, :dv].abs()
        o, l = p @ k[:, :dv], torch.logsumexp(logits, -1)
        tol = 2.0 ** -8 * (o.abs() + A) * (1 + 2.0 ** -7) + 2 * X * A + 1e-30
        ltol = X[:, 0] + 2.0 ** -22 * (1 + l.abs())
        parts.append([z.view(count, H, -1).cpu() if z.dim() == 2 else z.view(count, H).cpu() for z in (o, l, tol, ltol)])
        t += count
    return [torch.cat(z) for z in zip(*parts)]


@pytest.mark.parametrize("counts,lens,H,page,dv,dr,empty", [
    ([700, 500, 650, 333], [1200, 500, 901, 2000], 32, 64, 512, 64, 0),
    ([400, 391], [1500, 391], 20, 16, 512, 64, 0),
    ([1300], [1300], 33, 128, 256, 0, 0),
    ([300, 260], [1111, 255], 32, 32, 512, 64, 600),                   # 32-row tiles: most sequences are empty
])
def test_attn_many_row_tiles_of_a_sequence(counts, lens, H, page, dv, dr, empty):
    """Long causal chunks: several row tiles of a sequence for each SM, of different numbers of key tiles."""
    c = Cache(lens, page, dv + dr, seed=H)
    if empty:
        c.lens = torch.cat([c.lens, torch.zeros(empty, dtype=torch.int32)])
        c.table = torch.cat([c.table, torch.full((empty, c.table.shape[1]), -1, dtype=torch.int32)])
        counts = counts + [0] * empty
    q, out, lse, scale = run_attn(c, counts, H, dv, varlen=True)
    assert kda.kda_get_device_error() == 0
    ref = oracle_on_gpu(q, c.keys, counts, dv, scale)
    check_attn(out, lse, ref)


@pytest.mark.parametrize("T,H,d,rot,offset,dtype", [(8195, 3, 64, 32, 16, torch.bfloat16), (2051, 2, 96, 96, 0, torch.float32),
                                                    (7, 33, 576, 64, 512, torch.float32), (4100, 1, 16, 16, 0, torch.bfloat16)])
def test_rope_blocks_of_several_tokens_and_shares_of_heads(T, H, d, rot, offset, dtype):
    x = torch.randn(T, H, d, generator=gen(T)).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=gen(T + 1), dtype=torch.int32)
    f = freqs_of(rot)
    y = kda.kda_rope(x.to(DEV), pos.to(DEV), f.to(DEV), offset=offset)
    part = x[..., offset:offset + rot]
    check_rotated(y[..., offset:offset + rot], part, rotate64(part, pos, f, False), False, 1.0)
    keep = torch.ones(d, dtype=torch.bool)
    keep[offset:offset + rot] = False
    assert torch.equal(y.cpu()[..., keep], x[..., keep])


@pytest.mark.parametrize("T,H", [(1026, 5), (2200, 3)])
def test_append_blocks_of_several_tokens(T, H):
    """Blocks of 2 and 4 tokens, with rows behind the last sequence in the last one."""
    extra, page, dk, rot = 3, 32, 192, 64
    counts = [T // 3, 0, T - T // 3]
    lens = [counts[0] + 77, 5, counts[2]]
    c = Cache(lens, page, dk, seed=T)
    cache, table, ln = c.to_gpu()
    before = cache.clone()
    kv = torch.randn(T + extra, dk, generator=gen(1)).to(torch.bfloat16)
    q_pe = torch.randn(T + extra, H, rot, generator=gen(2)).to(torch.bfloat16)
    q = torch.full((T + extra, H, dk), 7.0, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, counts[0], counts[0], T], dtype=torch.int32, device=DEV)
    f = freqs_of(rot)
    kda.kda_latent_append(kv.to(DEV), cache, table, ln, q_pe=q_pe.to(DEV), q=q, freqs=f.to(DEV), cu_seqlens=cu)
    assert kda.kda_get_device_error() == 0
    seq = torch.tensor([0] * counts[0] + [2] * counts[2])
    pos = torch.cat([torch.arange(counts[0]) + 77, torch.arange(counts[2])])
    ids, rows = c.table[seq, pos // page].long(), pos % page
    got = cache[ids.to(DEV), rows.to(DEV)].cpu()
    assert torch.equal(got[:, :dk - rot], kv[:T, :dk - rot])
    part = kv[:T, None, dk - rot:]
    check_rotated(got[:, None, dk - rot:], part, rotate64(part, pos, f, False), False, 1.0)
    check_rotated(q[:T, :, dk - rot:], q_pe[:T], rotate64(q_pe[:T], pos, f, False), False, 1.0)
    assert (q[T:] == 7).all() and (q[..., :dk - rot] == 7).all()
    before[ids.to(DEV), rows.to(DEV)] = got.to(DEV)                    # nothing else was written
    assert torch.equal(torch.nan_to_num(cache.float(), 123.0), torch.nan_to_num(before.float(), 123.0))


# ------------------------------------------------------------------ a step as a graph
def test_a_captured_step_of_all_calls():
    """Fork, append, attention, compaction and a rotation in one graph, replayed on
    other inputs, beside the same calls made eagerly on copies."""
    H, dk, page, N = 4, 576, 16, 3
    i32 = dict(dtype=torch.int32, device=DEV)
    f = freqs_of(64).to(DEV)

    def inputs(seed):
        g = gen(seed)
        lens = torch.randint(17, 48, (N,), generator=g, dtype=torch.int32)
        table = torch.full((N, 3), -1, dtype=torch.int32)
        ids = torch.randperm(20, generator=g)[:9].int().view(N, 3)
        for n in range(N):
            table[n, :-(-int(lens[n]) // page)] = ids[n, :-(-int(lens[n]) // page)]
        # the first sequence's last page is copied to a free one, and named by its table
        last = (int(lens[0]) - 1) // page
        free = [i for i in range(20) if i not in ids.flatten().tolist()][0]
        src, dst = table[0, last:last + 1].clone(), torch.tensor([free], dtype=torch.int32)
        table[0, last] = free
        return [torch.randn(20, page, dk, generator=g).to(torch.bfloat16), table, lens, src, dst,
                torch.randn(N, dk, generator=g).to(torch.bfloat16), torch.randn(N, H, dk, generator=g).to(torch.bfloat16)]

    def step(cache, table, lens, src, dst, kv, q):
        kda.kda_pages_copy(cache, src, dst)
        kda.kda_latent_append(kv, cache, table, lens, q_pe=q[..., 512:], q=q, freqs=f)
        a = kda.kda_latent_attn(q, cache, table, lens, scale=0.07)
        kda.kda_pages_compact(cache, table, out=table)
        b = kda.kda_latent_attn(q, cache, table, lens, scale=0.07)
        return [*a, *b, kda.kda_rope(q, lens, f, offset=512, inverse=True)]

    held = [x.to(DEV) for x in inputs(0)]
    step(*[x.clone() for x in held])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step(*held)
    for seed in range(1, 9):
        new = [x.to(DEV) for x in inputs(seed)]
        for h, x in zip(held, new):
            h.copy_(x)
        graph.replay()
        eager = step(*new)
        torch.cuda.synchronize()
        assert kda.kda_get_device_error() == 0
        assert all(torch.equal(a, b) for a, b in zip(made, eager))
        assert torch.equal(held[1], new[1]) and int(held[1].max()) < int((held[1] >= 0).sum())
        # the attention is the same before and after its pages have moved
        assert torch.equal(made[0], made[2]) and torch.equal(made[1], made[3])
        live = held[1][held[1] >= 0].long()
        assert torch.equal(held[0][live], new[0][live])


def test_calls_of_every_kind_from_two_threads():
    """Appends, rotations, copies and compactions at once: each thread's own buffers come out as they do alone."""
    f = freqs_of(64).to(DEV)

    def job(seed):
        g = gen(seed)
        i32 = dict(dtype=torch.int32, device=DEV)
        cache = torch.randn(40, 16, 576, generator=g).to(DEV, torch.bfloat16)
        kv, q = torch.randn(6, 576, generator=g).to(DEV, torch.bfloat16), torch.randn(6, 8, 576, generator=g).to(DEV, torch.bfloat16)
        table = torch.randperm(40, generator=g)[:12].int().view(2, 6).to(DEV)
        lens = torch.tensor([70, 33], **i32)
        src, dst = torch.randperm(40, generator=g)[:30].int().to(DEV), torch.randperm(40, generator=g)[:30].int().to(DEV)

        def once():
            c, p = cache.clone(), q.clone()
            kda.kda_latent_append(kv, c, table, lens, q_pe=p[..., 512:], q=p, freqs=f)
            kda.kda_pages_copy(c, src, dst)
            names = kda.kda_pages_compact(c, table)
            return c[names.long()], p, names, kda.kda_rope(p, torch.arange(6, **i32), f, offset=8)

        want = once()
        torch.cuda.synchronize()
        return lambda: None if all(torch.equal(a, b) for a, b in zip(once(), want)) else "another answer"

    assert not both_at_once([job(1), job(2)])
    assert kda.kda_get_device_error() == 0
