"""The operators on a paged cache where sequences share pages, where calls run
on several streams, and at the ends of their arguments' ranges.  References are
64-bit computations; the tolerances are those of test_paged_gpu.py, which
derives them, unless a test says otherwise."""
import math
import random

import pytest
import torch

import dense_gemm_transformer_gb300 as dg
from tests.test_paged_gpu import BF16, FP16, FP32, Case, Model, _cache, _gen, _i32, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    dg.load(build_if_missing=True)
    handle = dg.Gemm()
    yield handle
    handle.close()


# ------------------------------------------------------- pages that are shared

class OwnPages(Model):
    """Model, with a sequence that appends to a page another one holds given its own copy of it (with pools), or
    refused (without)."""

    def shared(self, s, c):
        return c > 0 and self.lens[s] % self.page != 0 and self.refs[self.rows[s][-1]] > 1

    def grow(self, seqs, counts, pools=True):
        own = [self.shared(s, c) for s, c in zip(seqs, counts)]
        want = [self.need(self.lens[s] + c) - self.need(self.lens[s]) + o for s, c, o in zip(seqs, counts, own)]
        missing = max(0, sum(want) - len(self.free()))
        refused = sum(self.lens[s] + c > self.width * self.page or (o and not pools)
                      for s, c, o in zip(seqs, counts, own))
        positions = [self.lens[s] + i for s, c in zip(seqs, counts) for i in range(c)]
        if missing or refused:
            return positions, [-1] * len(positions), [0, missing, refused], []
        slots, free, moves = [], self.free(), []
        for s, c, w, o in zip(seqs, counts, want, own):
            for i in range(w):
                p = free.pop(0)
                self.refs[p] = 1
                if o and i == 0:
                    moves.append((self.rows[s][-1], p))
                    self.refs[self.rows[s][-1]] -= 1
                    self.rows[s][-1] = p
                else:
                    self.rows[s].append(p)
            for t in range(self.lens[s], self.lens[s] + c):
                slots.append(self.rows[s][t // self.page] * self.page + t % self.page)
            self.lens[s] += c
        return positions, slots, [sum(want), 0, 0], moves


@pytest.mark.parametrize("sequences,width,page,pages,seed", [(6, 5, 16, 14, 6), (40, 30, 16, 300, 1), (9, 7, 3, 24, 2),
                                                              (30, 600, 32, 9000, 3), (1500, 4, 16, 5000, 4)])
@pytest.mark.parametrize("pools", [True, False])
def test_no_page_is_written_by_two_sequences(h, sequences, width, page, pages, seed, pools):
    """Random growing, shrinking into shared pages, forking and compacting against plain Python, every sequence's
    tokens written where grow says and read back through the table."""
    rng = random.Random(seed)
    m = OwnPages(sequences, width, page, pages)
    table, lens, refs = _cache(sequences, width, pages)
    pool = torch.full((pages, page, 1, 4), -1, dtype=torch.int32, device="cuda")
    extra = torch.arange(2 * pages, dtype=torch.int32, device="cuda").view(2, pages, 1).repeat(1, 1, 4 * page)
    mirror = extra.clone()
    text = [[] for _ in range(sequences)]  # what each sequence's tokens should hold
    stamp, copies = 0, 0

    def follow(moves):
        if moves:
            src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
            mirror[:, dst] = mirror[:, src]

    for step in range(60):
        what = rng.choice(["grow", "grow", "shrink", "shrink", "fork", "fork", "compact"])
        if what == "grow":
            seqs = rng.sample(range(sequences), rng.randint(1, min(sequences, 300)))
            counts = [rng.choice([0, 1, 1, page, rng.randint(0, page * min(width, 6) // 2)]) for _ in seqs]
            if rng.random() < 0.5:  # few refusals for want of room
                counts = [min(c, width * page - m.lens[s]) for s, c in zip(seqs, counts)]
            positions, slots, info, moves = m.grow(seqs, counts, pools)
            copies += len(moves)
            got = h.cache_grow(table, lens, refs, page, _i32(seqs), _i32(counts), sum(counts),
                               pools=(pool, extra) if pools else None)
            assert got[0].tolist() == positions and got[1].tolist() == slots and got[2].tolist() == info
            follow(moves)
            if info[1:] == [0, 0] and slots:
                values = list(range(stamp, stamp + len(slots)))
                stamp += len(slots)
                pool.flatten(0, 1)[got[1]] = _i32(values)[:, None, None]
                for s, c in zip(seqs, counts):
                    text[s] += values[:c]
                    values = values[c:]
        elif what == "shrink":
            seqs = rng.sample(range(sequences), rng.randint(1, sequences // 2))
            counts = None if rng.random() < 0.1 else [rng.randint(0, page + 3) for _ in seqs]
            m.shrink(seqs, counts)
            h.cache_shrink(table, lens, refs, page, _i32(seqs), None if counts is None else _i32(counts))
            for s in seqs:
                del text[s][m.lens[s]:]
        elif what == "fork":
            empty = [s for s in range(sequences) if m.lens[s] == 0]
            held = [s for s in range(sequences) if m.lens[s] > 0]
            children = empty[:rng.randint(0, len(empty))]
            if not children or not held:
                continue
            parents = [rng.choice(held) for _ in children]
            copied, info, moves = m.fork(parents, children)
            got = h.cache_fork((pool, extra), table, lens, refs, page, _i32(parents), _i32(children))
            assert got[0].tolist() == copied and got[1].tolist() == info
            follow(moves)
            if info[1:] == [0, 0]:
                for p, c in zip(parents, children):
                    text[c] = list(text[p])
        else:
            info, moves = m.compact()
            assert h.cache_compact((pool, extra), table, refs).tolist() == info
            follow(moves)
        m.check(table, lens, refs)
        assert torch.equal(extra, mirror)
        rows, host = table.tolist(), pool[:, :, 0, 0].tolist()
        for s in range(sequences):
            assert text[s] == [host[rows[s][t // page]][t % page] for t in range(m.lens[s])], (step, s)
    assert h.check_device() == 0
    assert copies > 0 or not pools


@pytest.mark.parametrize("who", ["child", "parent", "both"])
def test_writing_after_a_shrink_leaves_the_other_sequence_as_it_was(who):
    """Fork, give tokens back into a page that is shared, append others: attention of both against their own keys."""
    heads, dim, page = 4, 64, 16
    cache = dg.PagedCache(2, 12, page, heads, dim, 2, 4, BF16)
    g = _gen(3)
    keys = {0: [], 1: []}

    def append(seqs, n):
        x = _randn(g, (len(seqs) * n, 3 * heads, dim), FP32)
        q, k, v = x.split(heads, 1)
        positions, slots, info = cache.grow(_i32(seqs), _i32([n] * len(seqs)), len(seqs) * n)
        assert info.tolist()[1:] == [0, 0] and int(slots.min()) >= 0
        assert int(cache.refs[slots // page].max()) == 1  # nobody else's page
        for layer in range(2):
            q16 = cache.append(layer, q, k, v, positions, slots)
        for i, s in enumerate(seqs):
            at = slice(i * n, (i + 1) * n)
            keys[s] += list(zip(k[at].to(BF16), v[at].to(BF16)))
        return q16

    append([0], 32)
    cache.fork(_i32([0]), _i32([1]))
    keys[1] = list(keys[0])
    grown = [1] if who == "child" else [0] if who == "parent" else [0, 1]
    cache.shrink(_i32(grown), _i32([3] * len(grown)))
    for s in grown:
        del keys[s][-3:]
    append(grown, 3)
    q = _randn(g, (2, heads, dim), BF16)
    for layer in range(2):
        out, lse = cache.attention(layer, q, return_lse=True)
        c = Case.__new__(Case)
        c.heads = c.kv_heads = heads
        c.dim, c.q, c.lengths = dim, q, [(1, 32), (1, 32)]
        c.keys, c.values = ([torch.stack([kv[i] for kv in keys[s]]) for s in (0, 1)] for i in (0, 1))
        c.check(out, lse)
    assert dg.default_handle().check_device() == 0


def test_a_shared_page_without_pools_is_refused(h):
    table, lens, refs = _cache(2, 4, 9)
    h.cache_grow(table, lens, refs, 16, _i32([0]), _i32([32]), 32)
    h.cache_fork((), table, lens, refs, 16, _i32([0]), _i32([1]))
    h.cache_shrink(table, lens, refs, 16, _i32([1]), _i32([5]))
    kept = table.clone(), lens.clone(), refs.clone()
    positions, slots, info = h.cache_grow(table, lens, refs, 16, _i32([1]), _i32([5]), 5)
    assert info.tolist() == [0, 0, 1] and slots.tolist() == [-1] * 5 and positions.tolist() == list(range(27, 32))
    for a, b in zip(kept, (table, lens, refs)):
        assert torch.equal(a, b)
    # no tokens, and a page that is full, need no copy
    assert h.cache_grow(table, lens, refs, 16, _i32([1, 0]), _i32([0, 2]), 2)[2].tolist() == [1, 0, 0]
    # the other holder gives the page up: it is the sequence's own again
    h.cache_shrink(table, lens, refs, 16, _i32([0]))
    assert h.cache_grow(table, lens, refs, 16, _i32([1]), _i32([5]), 5)[2].tolist() == [0, 0, 0]
    assert h.check_device() == 0


# -------------------------------------------------------- streams and handles

def test_cache_attention_gathers_on_the_stream_it_runs_on():
    """seqs and stream together: nothing of the call waits for the current stream, or runs on it."""
    cache = dg.PagedCache(1, 40, 16, 2, 64, 4, 16, BF16)
    seqs = torch.tensor([3, 1], device="cuda")
    positions, slots, info = cache.grow(_i32([0, 1, 2, 3]), _i32([50, 60, 70, 80]), 260)
    x = _randn(_gen(1), (260, 8, 64), FP32)
    cache.append(0, x[:, :4], x[:, 4:6], x[:, 6:], positions, slots)
    q = _randn(_gen(2), (2, 4, 64), BF16)
    want = cache.attention(0, q, seqs)
    side, raw = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    host = torch.empty(want.shape, dtype=BF16, pin_memory=True)
    for stream, given in ((side, side), (raw, raw.cuda_stream)):
        cache.attention(0, q, seqs, stream=given)  # (its memory is allocated)
        torch.cuda.synchronize()
        host.zero_()
        busy = torch.cuda.Event()
        torch.cuda._sleep(10 ** 9)
        busy.record()
        got = cache.attention(0, q, seqs, stream=given)
        stream.synchronize()
        assert not busy.query()  # the current stream has not come that far
        with torch.cuda.stream(stream):
            host.copy_(got, non_blocking=True)
        stream.synchronize()
        assert not busy.query()
        torch.cuda.synchronize()
        assert torch.equal(host, want.cpu())


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_belong_to_the_stream_of_the_call(h, raw):
    """A new output comes from the memory of the call's stream: never a block that work of the current stream, not
    yet run, still uses."""
    c = Case([(1, 40)] * 64, 4, 2, 64, 16, BF16, seed=1)
    freqs, _ = dg.rotary_frequencies(64, device="cuda")
    positions = torch.arange(64, device="cuda")
    table, lens, refs = _cache(3, 9, 30)
    seqs, counts = _i32([0, 2]), _i32([20, 33])
    side = torch.cuda.Stream()
    given = side.cuda_stream if raw else side
    torch.cuda.synchronize()

    def stream_of(t):
        at = t.data_ptr()
        return next(s["stream"] for s in torch.cuda.memory_snapshot()
                    if s["address"] <= at < s["address"] + s["total_size"])

    for call in (lambda s: h.paged_attention(c.q, c.k, c.v, c.table, c.lens, return_lse=True, stream=s),
                 lambda s: h.rotary(c.q, c.q, positions, freqs, stream=s),
                 lambda s: (h.rotary_append(c.q[:1], c.q[:1, :2], c.q[:1, :2], None, positions[:1], c.k, c.v, stream=s),),
                 lambda s: h.cache_grow(table, lens, refs, 16, seqs, counts, 53, stream=s)):
        for t in call(given):
            assert stream_of(t) == side.cuda_stream
        for t in call(None):
            assert stream_of(t) == torch.cuda.current_stream().cuda_stream
        torch.cuda.synchronize()
    assert h.check_device() == 0


def test_one_handle_on_several_streams(h):
    """Calls whose parts and counters live in the handle, at the same time on four streams: each as it is alone."""
    cases = [Case([(1, 9000 + 500 * i), (1, 300)], 12, 2, 128, 16, BF16, seed=i) for i in range(2)]
    cases += [Case([(150, 2500 + 300 * i), (2, 900)], 8, 2, 64, 16, FP16, seed=5 + i) for i in range(2)]
    want = [tuple(t.clone() for t in c.run(h)) for c in cases]
    assert h.plan()["split_k"] > 1
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(40):
        for c, s, g in zip(cases, streams, got):
            g.append(c.run(h, stream=s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for out, lse in g:
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
    # and afterwards
    for c, w in zip(cases, want):
        assert torch.equal(c.run(h)[0], w[0])
    assert h.check_device() == 0


def test_page_management_on_several_streams(h):
    streams = [torch.cuda.Stream() for _ in range(3)]
    states = []
    for i in range(3):
        table, lens, refs = _cache(40, 50, 60000 + 5000 * i)
        states.append((table, lens, refs, Model(40, 50, 16, 60000 + 5000 * i)))
    torch.cuda.synchronize()
    for step in range(20):
        got = []
        for i, ((table, lens, refs, m), s) in enumerate(zip(states, streams)):
            seqs, counts = list(range(step % 7, 40, 2 + i)), []
            counts = [1 + (step * 7 + x) % 30 for x in seqs]
            a, b = _i32(seqs), _i32(counts)
            torch.cuda.current_stream().synchronize()
            got.append((h.cache_grow(table, lens, refs, 16, a, b, sum(counts), stream=s), seqs, counts, a, b))
        torch.cuda.synchronize()
        for (table, lens, refs, m), ((positions, slots, info), seqs, counts, _, _) in zip(states, got):
            want = m.grow(seqs, counts)
            assert positions.tolist() == want[0] and slots.tolist() == want[1] and info.tolist() == want[2]
    for table, lens, refs, m in states:
        m.check(table, lens, refs)
    assert h.check_device() == 0


@pytest.mark.parametrize("lengths", [[(1, 3000)] * 3, [(130, 4000), (1, 50)]])
def test_a_first_call_can_be_captured(lengths):
    """A handle that has no scratch yet, in a graph."""
    handle = dg.Gemm()
    c = Case(lengths, 8, 2, 64, 16, BF16, seed=6)
    out = torch.zeros_like(c.q)
    table, lens, refs = _cache(3, 9, 30)
    seqs, counts = _i32([0, 2]), _i32([20, 33])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        handle.paged_attention(c.q, c.k, c.v, c.table, c.lens, cu_q=c.cu, max_q=c.max_q, out=out)
        grown = handle.cache_grow(table, lens, refs, 16, seqs, counts, 53)
    for _ in range(3):
        lens.zero_(), refs.zero_(), table.fill_(-1), out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = c.run(handle)[0]
        assert torch.equal(out, want)
        m = Model(3, 9, 16, 30)
        assert [t.tolist() for t in grown] == list(m.grow([0, 2], [20, 33]))
        m.check(table, lens, refs)
    assert handle.check_device() == 0
    del graph
    torch.cuda.synchronize()
    handle.close()


def test_a_handle_of_another_device_is_refused(h):
    """The check comes before anything else of a handle is read: a handle that is its first word, the device, and
    zeros, is refused by every call."""
    import ctypes
    from tests import test_paged_host as host
    lib = dg.load()
    fake = (ctypes.c_int32 * 4096)(torch.cuda.current_device() + 1)
    handle = ctypes.cast(fake, ctypes.c_void_p)
    assert lib.gemm_rotary(handle, host._pack("gemm_rotary_t", host.ROTARY), None) == host.INVALID
    attention = {**host.ATTENTION, "out": host.P + 0x100000}
    assert lib.gemm_paged_attention(handle, host._pack("gemm_paged_attention_t", attention), None) == host.INVALID
    c, p = host._cache(), host.P
    assert lib.gemm_cache_grow(handle, c, 1, p, p, 1, p, p, p, None) == host.INVALID
    assert lib.gemm_cache_shrink(handle, c, 1, p, p, None) == host.INVALID
    assert lib.gemm_cache_fork(handle, c, 1, p, p, p, p, None) == host.INVALID
    assert lib.gemm_cache_compact(handle, c, p, None) == host.INVALID
    assert lib.gemm_cache_copy(handle, c, 1, p, p, None) == host.INVALID


# ------------------------------------------------------------------- soft caps

@pytest.mark.parametrize("lengths", [[(1, 700), (1, 5)], [(20, 333)], [(150, 903), (40, 41)]])
@pytest.mark.parametrize("softcap", [0.5, 63.0, 65.0, 1e3, 1e4, 1e6, 1e8, 1e20, 1e30, 3e38])
def test_attention_caps_of_any_size(h, lengths, softcap):
    """A score through a cap is as exact as one without: the error grows with min(|s|, c), not with c.  With x = s / c
    the tanh is off by 2^-21 of itself where its form does not cancel (two units of 2^-24 in its own value and as
    many in x) and, up to a cap of 64, by 2^-21 c at most."""
    c = Case(lengths, 4, 2, 128, 16, BF16, seed=18)
    out, lse = c.run(h, softcap=softcap)
    start = 0
    for b, (n, length) in enumerate(lengths):
        q = c.q[start:start + n].double().transpose(0, 1)
        k, v = (t.double().transpose(0, 1).repeat_interleave(2, 0) for t in (c.keys[b], c.values[b]))
        seen = torch.arange(length, device="cuda") <= length - n + torch.arange(n, device="cuda")[:, None]
        s = q @ k.transpose(1, 2) / math.sqrt(128)
        mag = (q.abs() @ k.abs().transpose(1, 2) / math.sqrt(128)).masked_fill(~seen, 0).amax(-1, keepdim=True)
        s = softcap * torch.tanh(s / softcap)
        form = 2.0 ** -21 * torch.minimum(mag, torch.tensor(float(softcap)).double()) if softcap > 64 else 2.0 ** -21 * softcap
        delta = 2.0 ** -22 * (128 / 16 + 2) * mag + form + 2.0 ** -21
        w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
        ref, scale_w = w @ v, w @ v.abs()
        ref_lse = torch.logsumexp(s.masked_fill(~seen, -math.inf), -1)
        bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 4 * delta + 2.0 ** -20) * scale_w + 2.0 ** -24
        err = (out[start:start + n].double().transpose(0, 1) - ref).abs()
        assert bool((err <= bound).all()), (b, float((err / bound).max()))
        err = (lse[start:start + n].double().transpose(0, 1) - ref_lse).abs()
        bound = 2 * delta[..., 0] + 2.0 ** -21 * (1 + ref_lse.abs())
        assert bool((err <= bound).all()), (b, "lse", float((err / bound).max()))
        start += n
    assert h.check_device() == 0


def test_attention_capped_with_a_scale_of_zero(h):
    """All scores are 0: every row is the mean of what it sees, in the time of any other scale.  (The mean of numbers
    that the products take exactly: only the sums, 2^-20, and the result are rounded.)"""
    c = Case([(1000, 3000)], 16, 2, 128, 16, BF16, seed=4)
    time = {}
    for scale in (0.0, 0.1):
        for _ in range(3):
            out, lse = c.run(h, softcap=30.0, scale=scale)
        began, ended = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        began.record()
        for _ in range(5):
            c.run(h, softcap=30.0, scale=scale)
        ended.record()
        torch.cuda.synchronize()
        time[scale] = began.elapsed_time(ended)
    assert time[0.0] < 3 * time[0.1], time
    c.check(*c.run(h, softcap=30.0, scale=0.0), 0.0, 30.0)
    assert h.check_device() == 0


def test_attention_offsets_out_of_order_leave_the_other_sequences(h):
    """Overlapping ranges of tokens with offsets out of order between them: more work than the call has room for is
    reported and left out, what comes before it is right, whatever the call before had."""
    small = Case([(40, 60)], 4, 2, 128, 16, BF16, seed=1)
    c = Case([(100, 3000)] + [(1000, 1000)], 4, 2, 128, 16, BF16, seed=2)
    table = torch.cat([c.table[:1]] + [c.table[1:]] * 31)
    lens = torch.cat([c.lens[:1]] + [c.lens[1:]] * 31)
    cu = _i32([0, 100] + [1100, 100] * 15 + [1100])
    assert cu.numel() == table.shape[0] + 1
    small.run(h)
    out, lse = h.paged_attention(c.q, c.k, c.v, table, lens, cu_q=cu, max_q=1000, return_lse=True)
    assert h.check_device() == 8
    assert h.plan()["split_k"] > 1
    first = Case.__new__(Case)
    first.__dict__.update(c.__dict__)
    first.lengths, first.keys, first.values, first.q = c.lengths[:1], c.keys[:1], c.values[:1], c.q[:100]
    first.check(out[:100], lse[:100])


def test_out_of_memory_is_torch_s_own_error(h):
    q = torch.zeros(1, 1, 64, device="cuda").expand(2 ** 24, 2 ** 10, 64)  # 4 TiB of output
    freqs, _ = dg.rotary_frequencies(64, device="cuda")
    positions = torch.zeros(2 ** 24, dtype=torch.int64, device="cuda")
    with pytest.raises(torch.cuda.OutOfMemoryError):
        h.rotary(q, None, positions, freqs)
    assert h.check_device() == 0


# ------------------------------------------------------------------- pages

# ------------------------------------------------------------ tables that are wrong

def test_compact_leaves_an_entry_of_a_free_page(h):
    """A table entry that names a page which refs calls free has no new place: reported, and left as it is."""
    table, lens, refs = _cache(3, 4, 40)
    pool = torch.arange(40, dtype=torch.int32, device="cuda").view(40, 1).repeat(1, 4)
    # scratch words of earlier calls
    h.cache_grow(table, lens, refs, 16, _i32([0, 1, 2]), _i32([64, 64, 64]), 192)
    h.cache_shrink(table, lens, refs, 16, _i32([0]))
    h.cache_compact((pool,), table, refs)
    table.fill_(-1), lens.zero_(), refs.zero_()
    refs[30], refs[35] = 1, 2
    table[0, 0], table[1, 0], table[2, 0] = 30, 35, 35
    table[2, 1] = 33  # free
    table[1, 1] = 10 ** 6
    info = h.cache_compact((pool,), table, refs)
    assert info.tolist() == [2, 2]
    assert table[:, :2].tolist() == [[0, -1], [1, 10 ** 6], [1, 33]]
    assert h.check_device() == 8


def test_grow_totals_beyond_32_bits(h):
    """More pages wanted than an int counts (by rows that are one row, repeated): missing, and nothing changed."""
    width = 2 ** 31 - 2 ** 17
    row = torch.empty(1, width, dtype=torch.int32, device="cuda")
    row[0, :8] = -1
    table = row.expand(6, width)
    lens, refs = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.zeros(5000, dtype=torch.int32, device="cuda")
    for counts in ([1_500_000_000] * 2, [1_500_000_000] * 3, [2_000_000_000] * 6, [1, 2_000_000_000, 2_000_000_000]):
        seqs = list(range(len(counts)))
        positions, slots, info = h.cache_grow(table, lens, refs, 1, _i32(seqs), _i32(counts), 4)
        assert info.tolist() == [0, min(sum(counts) - 5000, 2 ** 31 - 1), 0] and slots.tolist() == [-1] * 4
        assert h.check_device() == 8  # `tokens` is not the sum of the counts
    assert int(lens.abs().sum()) == 0 and int(refs.abs().sum()) == 0
    del row, table
    torch.cuda.empty_cache()


def test_append_of_no_tokens(h):
    """Nothing to append is no error, as nothing to rotate is not."""
    x = torch.empty(0, 4, 64, device="cuda")
    pools = [torch.ones(2, 16, 4, 64, dtype=BF16, device="cuda") for _ in range(2)]
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    freqs, _ = dg.rotary_frequencies(64, device="cuda")
    assert h.rotary_append(x, x, x, none, none, *pools, freqs).shape == x.shape
    assert h.rotary_append(x, x, x, None, none, *pools).dtype == BF16
    assert all(bool((p == 1).all()) for p in pools) and h.check_device() == 0


# --------------------------------------------- windows, values and small weights

@pytest.mark.parametrize("n,length", [(1, 5), (4, 1), (30, 10), (200, 60), (5, 300)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 30])
def test_attention_windows_beyond_every_key(h, n, length, window):
    """A window that no sequence fills is none, also where there are more new tokens than keys."""
    c = Case([(n, length), (1, 40)], 4, 2, 64, 16, BF16, seed=13)
    out, lse = c.run(h, window=window)
    c.check(out, lse, None, 0.0, 0)
    assert h.check_device() == 0


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_attention_many_small_weights(h, dtype):
    """Four keys far above a million others, whose weights of 2^-18 1.0078 each add up to as much: fp16 has no more
    than 8 bits for such a number.  So many sequences (of the same pages) that none is split, and the four where each
    warp of a block meets one."""
    dim, page, length, sequences = 64, 128, 2 ** 20, 1216
    k = torch.zeros(length // page, page, 1, dim, dtype=dtype, device="cuda")
    v = torch.ones_like(k)
    q = torch.zeros(sequences, 1, dim, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    k[0, 0:64:16, :, 0] = 1.0
    v[0, 0:64:16] = 0.0
    scale = (18 - math.log2(1.0078)) * math.log(2)
    table = torch.arange(length // page, dtype=torch.int32, device="cuda")[None].expand(sequences, -1)
    lens = torch.full((sequences,), length, dtype=torch.int32, device="cuda")
    out, lse = h.paged_attention(q, k, v, table, lens, scale=scale, return_lse=True)
    assert h.plan()["split_k"] == 1
    others = (length - 4) * math.exp(-scale)
    want = others / (4 + others)
    # the scale as an fp32 (2^-25 of 12.5) and the weights' function, 2^-20; the sums of a warp's quarter million keys,
    # 16 a product, at most 2^14 steps of 2^-24 (and half as much on average); the output's own rounding
    assert float((out.double() - want).abs().max()) <= want * (torch.finfo(dtype).eps / 2 + 2.0 ** -10)
    assert abs(float(lse[0, 0]) - (scale + math.log(4 + others))) <= 2.0 ** -10
    assert h.check_device() == 0


# --------------------------------------------- values, windows and other ends

@pytest.mark.parametrize("n,length", [(1, 1), (1, 700), (3, 60), (20, 333), (40, 300), (150, 400)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_attention_infinite_values_give_infinities(h, n, length, dtype):
    """A value of infinity that a row sees, with a weight above 0, makes its output that infinity, and one of each
    sign not a number; the other columns and heads are as they are without."""
    c = Case([(n, length)], 4, 2, 64, 16, dtype, seed=31)
    at = max(0, length - n - 2)  # seen by every row
    v = c.values[0][at].clone()
    clean, lse_clean = c.run(h)
    v[0, 3], v[0, 7] = math.inf, -math.inf
    c.put(0, at, v=v)
    out, lse = c.run(h)
    assert bool((out[:, :2, 3] == math.inf).all()) and bool((out[:, :2, 7] == -math.inf).all())
    rest = torch.ones(64, dtype=torch.bool, device="cuda")
    rest[[3, 7]] = False
    ref, bound, _, _ = next(c.reference(dtype))
    err = (out.double().transpose(0, 1) - ref).abs()
    assert bool((err <= bound)[:, :, rest].all())
    assert torch.equal(out[:, 2:], clean[:, 2:])
    if length > 4:
        v[0, 3] = math.inf
        c.put(0, at, v=v)
        other = c.values[0][at - 1].clone()
        other[0, 3] = -math.inf
        c.put(0, at - 1, v=other)
        out, _ = c.run(h)
        assert bool(out[:, :2, 3].isnan().all()) and bool((out[:, :2, 7] == -math.inf).all())
    assert h.check_device() == 0


def test_attention_in_place_is_refused(h):
    """out over q: rows may be computed a second time, from their queries."""
    c = Case([(40, 100)], 4, 2, 64, 16, BF16)
    q = c.q.contiguous()
    with pytest.raises(dg.GemmError, match="INVALID_VALUE"):
        h.paged_attention(q, c.k, c.v, c.table, c.lens, cu_q=c.cu, max_q=c.max_q, out=q)


@pytest.mark.parametrize("lengths", [[(1, 300)], [(100, 300), (1, 20)]])
def test_attention_broadcast_tensors(h, lengths):
    """Keys and values of one head expanded to several, queries of one head to several: strides of zero."""
    c = Case(lengths, 4, 1, 64, 16, BF16, seed=3)
    q = c.q[:, :1].expand(-1, 4, -1)
    kw = dict(cu_q=c.cu, max_q=c.max_q, return_lse=True)
    want = h.paged_attention(q.contiguous(), c.k, c.v, c.table, c.lens, **kw)
    got = h.paged_attention(q, c.k, c.v, c.table, c.lens, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k, v = (t.expand(-1, -1, 4, -1) for t in (c.k, c.v))
    c.q, c.kv_heads = q, 4
    c.keys, c.values = [t.expand(-1, 4, -1) for t in c.keys], [t.expand(-1, 4, -1) for t in c.values]
    c.check(*h.paged_attention(q, k, v, c.table, c.lens, **kw))
    assert h.check_device() == 0


@pytest.mark.parametrize("heads", [8, 258])
def test_attention_with_a_loose_bound_on_new_tokens(h, heads):
    """max_q is an upper bound; one far above the tokens there are changes nothing."""
    c = Case([(1, 30 + i) for i in range(50)] + [(3, 40)], heads, 2, 64, 16, BF16, seed=2)
    for c.max_q in (100, 2 ** 31 - 1):
        got = c.run(h)
        c.check(*got)
    assert h.check_device() == 0


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("lengths", [[(512, 4096)], [(1, 4096)] * 16])
def test_attention_time_with_values_that_are_not_finite(h, lengths, bad):
    """A value of every head that every row sees: all rows are computed again, which takes longer, not forever."""
    c = Case(lengths, 32, 4, 128, 64, BF16, seed=17)

    def time():
        c.run(h)
        began, ended = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        began.record()
        c.run(h)
        ended.record()
        torch.cuda.synchronize()
        return began.elapsed_time(ended)

    clean = min(time() for _ in range(3))
    for b in range(len(lengths)):
        c.put(b, 100, v=torch.full((4, 128), bad))
    out, lse = c.run(h)
    assert bool((out.isnan() if bad != bad else out == math.inf).all()) and bool(torch.isfinite(lse).all())
    spent = min(time() for _ in range(3))
    assert spent < 100 * clean + 1.0, (spent, clean)
    assert h.check_device() == 0
