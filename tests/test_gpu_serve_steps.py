"""Attention of chunks, rotary positions and log probabilities (include/wbserve.h) as a model's step uses
them: one after the other, captured and replayed with other lengths, on several streams at once, with
workspaces that hold anything, and past one launch's size."""
import math

import numpy as np
import pytest

from tests.test_gpu_serve_chunk import TYPES, check as check_chunk, rand, random_cache
from tests.test_gpu_serve_logprobs import run as check_logprobs
from tests.test_gpu_serve_rotate import check as check_rotated

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def i32(a):
    return torch.tensor(np.asarray(a, np.int32)).cuda()


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


class Layer:
    """A full-attention layer's buffers and its step on rows of a fused projection [N, (Hq + 2 H) D]."""

    def __init__(self, R, H, G, D, kv, qt, page, pages, width, N, seed):
        g = torch.Generator().manual_seed(seed)
        self.R, self.H, self.G, self.D, self.page, self.N, self.kv, self.qt = R, H, G, D, page, N, kv, qt
        self.k, self.ks = random_cache(g, pages, H, page, D, kv)
        self.v, self.vs = random_cache(g, pages, H, page, D, kv)
        self.table, self.free, self.n_free = i32(np.full((R, width), -1)), torch.randperm(pages, generator=g).int().cuda(), i32([pages])
        self.lens, self.starts, self.status, self.more = i32([0] * R), i32([0] * (R + 1)), i32([9]), i32([0] * R)
        self.slots = torch.empty(N, dtype=torch.int64, device="cuda")
        self.x = rand(g, N, (G * H + 2 * H) * D, dtype=qt).cuda()
        self.positions = i32([0] * N)
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=g)).to(TYPES[qt]).cuda() for _ in range(2))
        self.o = torch.full((N, G * H, D), 7.0, dtype=TYPES[qt], device="cuda")
        self.lse = torch.full((N, G * H), 7.0, device="cuda")
        self.head = (torch.randn((G * H * D, 5003), generator=g) / 8).to(TYPES[qt]).cuda()
        self.tokens = torch.randint(0, 5003, (N,), generator=g).cuda()
        self.lp, self.entropy = (torch.full((N,), 7.0, device="cuda") for _ in range(2))
        self.ids, self.top = torch.full((N, 5), -7, dtype=torch.int32, device="cuda"), torch.full((N, 5), 7.0, device="cuda")
        import linear_attn_decode_amd as wb
        self.freqs = wb.rotary_frequencies(D // 2, base=50000.0, factor=4.0, context=4096)
        q, kk, vv = self.x.split([G * H * D, H * D, H * D], 1)
        self.q, self.nk, self.nv = q.unflatten(1, (G * H, D)), kk.unflatten(1, (H, D)), vv.unflatten(1, (H, D))

    def step(self):
        import linear_attn_decode_amd as wb
        wb.plan_pages(self.lens, self.more, self.table, self.free, self.n_free, self.page, self.slots, self.starts, self.status)
        wb.qk_rotate(self.q, self.nk, self.positions, self.freqs, q_weight=self.qw, k_weight=self.kw, magnitude=1.25)
        wb.kv_append(self.nk, self.nv, self.k, self.v, self.slots, k_scale=self.ks, v_scale=self.vs)
        wb.kv_attend_chunk(self.q, self.k, self.v, self.table, self.lens, self.starts, self.o, lse=self.lse, k_scale=self.ks,
                           v_scale=self.vs)
        self.logits = self.o.flatten(1) @ self.head
        wb.token_logprobs(self.logits, self.tokens, self.lp, entropy=self.entropy, top_ids=self.ids, top_logprobs=self.top)

    def feed(self, g, more):
        """The next step's rows (padded to N), their positions and counts."""
        lens = self.lens.cpu().numpy()
        at = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, more)] + [np.zeros(self.N - sum(more))]).astype(np.int32)
        self.x.copy_(rand(g, *self.x.shape, dtype=self.qt))
        self.positions.copy_(torch.from_numpy(at))
        self.more.copy_(i32(more))
        return at


@pytest.mark.parametrize("kv,qt,D,H,G,page", [("bf16", "bf16", 128, 2, 4, 16), ("f16", "f16", 64, 3, 1, 8), ("e4m3", "bf16", 128, 1, 8, 64),
                                              ("bf16", "bf16", 256, 2, 2, 32)])
def test_a_layers_steps(kv, qt, D, H, G, page):
    """Prompts, parts of prompts, drafted and single tokens of four requests through plan_pages, qk_rotate (in place, on
    views of a fused projection), kv_append, kv_attend_chunk and token_logprobs, each step's outputs against the
    float64 definitions; a step of single tokens through kv_attend too."""
    import linear_attn_decode_amd as wb
    a = Layer(4, H, G, D, kv, qt, page, 400, 1200 // page, 320, 1)
    g = torch.Generator().manual_seed(2)
    for more in ([130, 1, 0, 63], [64, 4, 200, 5], [1, 1, 1, 1], [5, 0, 1, 300], [1, 1, 1, 1]):
        print(f"[step] {more}", flush=True)
        at = a.feed(g, more)
        before = a.x.clone()
        a.step()
        torch.cuda.synchronize()
        lens, starts, table, n = a.lens.cpu().tolist(), a.starts.cpu().tolist(), a.table.cpu().numpy(), sum(more)
        assert int(a.status) == 0 and starts[-1] == n
        old = before.split([G * H * D, H * D, H * D], 1)
        args = (1e-6, at, a.freqs.cpu().numpy(), False, 1.25)
        check_rotated(a.q, old[0].unflatten(1, (G * H, D)), a.qw, *args)
        check_rotated(a.nk, old[1].unflatten(1, (H, D)), a.kw, *args)
        assert torch.equal(bits(a.x[:, (G + 1) * H * D:]), bits(before[:, (G + 1) * H * D:]))
        s = a.slots[:n]
        if kv != "e4m3":
            for new, cache in ((a.nk, a.k), (a.nv, a.v)):
                assert torch.equal(bits(cache[s // page, :, s % page]), bits(new[:n].contiguous()))
        k64, v64 = (c.float().double().cpu().numpy() * (1 if sc is None else sc.double().cpu().numpy()[..., None])
                    for c, sc in ((a.k, a.ks), (a.v, a.vs)))
        check_chunk(a.o[:n], a.lse[:n], a.q[:n], k64, v64, table, lens, starts, page, 1 / math.sqrt(D), 0, kv, qt)
        if more == [1, 1, 1, 1]:
            one, lse = torch.empty_like(a.o[:4]), torch.empty((4, G * H), device="cuda")
            wb.kv_attend(a.q[:4], a.k, a.v, a.table, a.lens, one, lse=lse, k_scale=a.ks, v_scale=a.vs)
            torch.cuda.synchronize()
            check_chunk(one, lse, a.q[:4], k64, v64, table, lens, starts, page, 1 / math.sqrt(D), 0, kv, qt)
        rows = list(range(0, n, 41))
        got = check_logprobs(a.logits, a.tokens.cpu().tolist(), 5, rows=rows)
        for x, y in zip(got, (a.lp, a.entropy, a.ids, a.top)):
            assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("R,N", [(4, 320), (100, 500)])
def test_a_captured_layers_step_replays(R, N):
    """One graph of the step; counts, rows and positions change between replays."""
    a, b = (Layer(R, 2, 4, 128, "bf16", "bf16", 16, 3000, 100, N, 5) for _ in range(2))
    b.step()                                                 # (more is 0: nothing is stored)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.step()
    torch.cuda.synchronize()
    rng = np.random.default_rng(R)
    for step in range(6):
        more = [1] * R if step in (2, 5) else list(rng.multinomial(N if step % 2 else N - 7, rng.dirichlet(np.full(R, 0.3))))
        for s in (a, b):
            s.feed(torch.Generator().manual_seed(step), more)
            s.o.fill_(7.0)
            s.lse.fill_(7.0)
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        assert int(a.status) == 0
        n = sum(more)
        for name in ("k", "v", "table", "n_free", "lens", "starts", "x", "o", "lse", "lp", "entropy", "ids", "top"):
            x, y = getattr(a, name), getattr(b, name)
            if name in ("lp", "entropy", "ids", "top"):
                x, y = x[:n], y[:n]
            assert torch.equal(bits(x.contiguous()), bits(y.contiguous())), (name, step)
        assert (a.o[n:] == 7).all() and (a.lse[n:] == 7).all()
        float(a.o.float().sum())                             # eager work between the replays


def chunk_inputs(seed, R, m, width, H=2, G=4, D=128, page=16):
    g = torch.Generator().manual_seed(seed)
    k, v = (rand(g, 300, H, page, D, dtype="bf16").cuda() for _ in range(2))
    table = torch.randint(0, 300, (R, width), generator=g).int().cuda()
    q = rand(g, R * m, H * G, D, dtype="bf16").cuda()
    return q, k, v, table


@pytest.mark.parametrize("R,m,width", [(3, 5, 300), (20, 7, 100), (90, 3, 100), (5, 40, 10)])
def test_captured_chunks_replay_with_other_lengths(R, m, width):
    """Split and joined or not, requests counted in a launch before or not: replays give the eager call's bits."""
    import linear_attn_decode_amd as wb
    q, k, v, table = chunk_inputs(R, R, m, width)
    rng = np.random.default_rng(R)
    lens, starts = i32([m] * R), i32(np.arange(R + 1) * m)
    outs = [(torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")) for _ in range(2)]
    call = lambda o: wb.kv_attend_chunk(q, k, v, table, lens, starts, o[0], lse=o[1])
    call(outs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[1])
        call(outs[1])                                        # (in the first one's workspace, perhaps)
    most = width * 16
    for step in range(6):
        news = np.full(R, m) if step % 2 else rng.multinomial(R * m - step, np.full(R, 1 / R))
        n = np.minimum(news + [rng.integers(0, most, R), np.full(R, most), np.zeros(R, int), np.where(np.arange(R) == 1, most, 0),
                               rng.integers(0, 100, R), rng.integers(0, most, R)][step], most)
        lens.copy_(i32(n))
        starts.copy_(i32(np.concatenate([[0], np.cumsum(news)])))
        for o in outs:
            o[0].fill_(7.0)
            o[1].fill_(7.0)
        call(outs[0])
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(*outs):
            assert torch.equal(bits(x), bits(y)), step
        assert (outs[0][0][int(news.sum()):] == 7).all()
        q.copy_(torch.randn(q.shape, device="cuda").to(q.dtype))


def test_two_captured_graphs_replay_side_by_side():
    """Two graphs of chunks and log probabilities on other inputs, replayed on two streams at once."""
    import linear_attn_decode_amd as wb
    runs = []
    for i in range(2):
        q, k, v, table = chunk_inputs(40 + i, 6, 4, 200)
        lens, starts = i32([3200 - 100 * i, 40, 700, 9, 2000, 64]), i32(np.arange(7) * 4)
        x, t = torch.randn((2, 90000 + 8 * i), device="cuda"), torch.tensor([1, 70000]).cuda()

        def call(o, q=q, k=k, v=v, table=table, lens=lens, starts=starts, x=x, t=t):
            wb.kv_attend_chunk(q, k, v, table, lens, starts, o[0])
            wb.token_logprobs(x, t, o[1], top_ids=o[2], top_logprobs=o[3])
        outs = [(torch.empty_like(q), torch.empty(2, device="cuda"), torch.empty((2, 9), dtype=torch.int32, device="cuda"),
                 torch.empty((2, 9), device="cuda")) for _ in range(2)]
        call(outs[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                call(outs[1])
        runs.append((graph, call, outs, torch.cuda.Stream()))
    for _ in range(10):
        for _, _, outs, _ in runs:
            for o in outs[1]:
                o.zero_()
        torch.cuda.synchronize()
        for graph, _, _, s in runs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, call, outs, _ in runs:
            for x, y in zip(*outs):
                assert torch.equal(bits(x), bits(y))
            call(outs[0])                                    # eager work between
        torch.cuda.synchronize()


def test_calls_on_two_streams_do_not_disturb_each_other():
    """The same calls on two streams at once, one made current and one passed."""
    import linear_attn_decode_amd as wb
    runs = []
    for i in range(2):
        q, k, v, table = chunk_inputs(50 + i, 3, 6, 250)
        lens, starts, x, t = i32([4000, 700 + i, 6]), i32(np.arange(4) * 6), torch.randn((1, 120000), device="cuda"), torch.tensor([5]).cuda()
        freqs, at = wb.rotary_frequencies(128), i32(np.arange(18) * 50)

        def call(o, stream=None, q=q, k=k, v=v, table=table, lens=lens, starts=starts, x=x, t=t, freqs=freqs, at=at):
            wb.qk_rotate(q, None, at, freqs, q_out=o[0], stream=stream)
            wb.kv_attend_chunk(o[0], k, v, table, lens, starts, o[1], stream=stream)
            wb.token_logprobs(x, t, o[2], entropy=o[3], stream=stream)
        outs = [(torch.empty_like(q), torch.empty_like(q), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")) for _ in range(2)]
        call(outs[0])
        runs.append((call, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for _, outs, _ in runs:
            for o in outs[1]:
                o.zero_()
        torch.cuda.synchronize()
        for n, (call, outs, s) in enumerate(runs):
            if n:
                call(outs[1], stream=s)
            else:
                with torch.cuda.stream(s):
                    call(outs[1])
        torch.cuda.synchronize()
        for _, outs, _ in runs:
            for x, y in zip(*outs):
                assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("R", [3, 70])
def test_workspaces_may_hold_anything(R):
    """Zeros, ones, noise, and what a call of other lengths left: equal results."""
    import linear_attn_decode_amd as wb
    from linear_attn_decode_amd import serve as S
    q, k, v, table = chunk_inputs(60, R, 4, 200)
    starts = i32(np.arange(R + 1) * 4)
    H, D, page = k.shape[1], k.shape[3], k.shape[2]
    lens = [i32(np.full(R, 3200)), i32(4 + np.arange(R) * 17 % 3000)]
    want = [torch.empty_like(q) for _ in lens]
    for o, ln in zip(want, lens):
        wb.kv_attend_chunk(q, k, v, table, ln, starts, o)
    torch.cuda.synchronize()
    H, D, page = k.shape[1], k.shape[3], k.shape[2]
    n = S._chunk_work(S.BF16, 300, H, page, D, 4 * R, R, q.shape[1], 200)
    assert n > 0
    c = S._desc.pack(k.data_ptr(), v.data_ptr(), 0, 0, 300, page, H, D, S.BF16)
    fills = [torch.zeros(n, dtype=torch.uint8), torch.full((n,), 255, dtype=torch.uint8), torch.randint(0, 256, (n,), dtype=torch.uint8)]
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    for fill in fills + [None]:
        for ln, w in zip(lens, want):
            if fill is not None:
                work.copy_(fill)
            o = torch.full_like(q, 7.0)
            status = S._fn["kv_attend_chunk"](c, q.data_ptr(), q.stride(0), q.stride(1), S.BF16, 4 * R, R, q.shape[1],
                                              table.data_ptr(), 200, ln.data_ptr(), starts.data_ptr(), D ** -0.5, 0, o.data_ptr(),
                                              None, work.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert status == 0 and torch.equal(bits(o), bits(w))


def test_more_workgroups_than_a_launch_holds():
    """4200 requests of one token over 4096 key-value heads: 2^24 blocks of rows and more, of 256 lanes. Each row
    sees one token, whose value it has."""
    import linear_attn_decode_amd as wb
    R, H, D = 4200, 4096, 64
    g = torch.Generator().manual_seed(7)
    k, v = (rand(g, 3, H, 8, D, dtype="bf16").cuda() for _ in range(2))
    q = rand(g, 1, H, D, dtype="bf16").cuda().expand(R, H, D)
    o = torch.full((R, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(R, dtype=torch.int32, device="cuda")
    wb.kv_attend_chunk(q, k, v, (at % 3).view(R, 1), i32([1] * R), i32(np.arange(R + 1)), o)
    torch.cuda.synchronize()
    for p in range(3):
        assert (o[p::3] == v[p, :, 0]).all()


def test_outputs_past_the_caches():
    """Results of a call whose outputs are larger than the last-level cache: those of calls on parts of the rows."""
    import linear_attn_decode_amd as wb
    N, H, D = 30011, 40, 128
    x = torch.randn((N, H, D), device="cuda").bfloat16()
    assert 2 * x.numel() > 256 << 20
    at, freqs = torch.randint(0, 100000, (N,), device="cuda"), wb.rotary_frequencies(D)
    w = torch.rand(D, device="cuda").bfloat16()
    y, z = torch.empty_like(x), torch.empty_like(x)
    wb.qk_rotate(x[:, :32], x[:, 32:], at, freqs, q_weight=w, k_weight=w, q_out=y[:, :32], k_out=y[:, 32:])
    for i in range(0, N, 3000):
        r = slice(i, i + 3000)
        wb.qk_rotate(x[r, :32], x[r, 32:], at[r], freqs, q_weight=w, k_weight=w, q_out=z[r, :32], k_out=z[r, 32:])
    torch.cuda.synchronize()
    assert torch.equal(bits(y), bits(z))


def test_a_captured_rotation_follows_its_positions():
    import linear_attn_decode_amd as wb
    g = torch.Generator().manual_seed(8)
    x, at, freqs = rand(g, 9, 6, 96, dtype="f16").cuda(), i32([0] * 9), wb.rotary_frequencies(32, factor=8.0)
    y, z = torch.empty_like(x), torch.empty_like(x)
    call = lambda out: wb.qk_rotate(x, None, at, freqs, interleaved=True, q_out=out)
    call(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(z)
    for step in range(5):
        at.copy_(torch.randint(-100, 10 ** 6, (9,), generator=g).int())
        x.copy_(rand(g, 9, 6, 96, dtype="f16"))
        call(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(z)), step


def test_rows_of_logits_past_32_bits():
    """Logits whose byte and element offsets pass 2^32, rows far apart."""
    x = torch.zeros((3, 2 ** 31 + 1000), dtype=torch.bfloat16, device="cuda")[:, :5000]
    x.copy_(3 * torch.randn((3, 5000), generator=torch.Generator().manual_seed(9)))
    check_logprobs(x, [0, 4999, 17], 7)


def test_binding_refusals():
    """Every wrong argument is named, and nothing is launched."""
    import linear_attn_decode_amd as wb
    bf, f8, f32, f64, i, long = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.float64, torch.int32, torch.int64
    cu = lambda *a, dtype=bf: torch.zeros(*a, device="cuda").to(dtype)
    k, q, o = cu(4, 2, 16, 64), cu(5, 4, 64), cu(5, 4, 64)
    t, n, s = cu(3, 2, dtype=i), cu(3, dtype=i), cu(4, dtype=i)
    good = dict(q=q, k_cache=k, v_cache=k.clone(), table=t, lens=n, starts=s, o=o)
    host = lambda x: x.cpu()
    for match, kw in [("q, table: expected", dict(q=q[0])), ("q, table: expected", dict(table=n)), ("q, table: expected", dict(q=cu(5, 4, 64, dtype=i))),
                      ("q: expected", dict(q=cu(5, 4, 128))), ("q: expected", dict(q=host(q))), ("q: expected", dict(q=cu(5, 4, 128)[..., ::2])),
                      ("o: expected", dict(o=cu(5, 4, 128))), ("o: expected", dict(o=cu(4, 4, 64))), ("o: expected", dict(o=cu(5, 8, 64)[:, ::2])),
                      ("o: expected", dict(o=cu(5, 4, 64, dtype=f32))), ("table: expected", dict(table=t.long())),
                      ("table: expected", dict(table=cu(3, 4, dtype=i)[:, ::2])), ("lens: expected", dict(lens=s)), ("lens: expected", dict(lens=n.long())),
                      ("starts: expected", dict(starts=n)), ("starts: expected", dict(starts=host(s))), ("lse: expected", dict(lse=cu(5, 4))),
                      ("lse: expected", dict(lse=cu(4, 5, dtype=f32))), ("out of range", dict(window=-1)), ("v_cache: expected", dict(v_cache=cu(4, 2, 8, 64))),
                      ("k_scale, v_scale: only", dict(k_scale=cu(4, 2, 16, dtype=f32), v_scale=cu(4, 2, 16, dtype=f32))),
                      ("k_scale, v_scale: a float8", dict(k_cache=k.to(f8), v_cache=k.to(f8)))]:
        with pytest.raises(ValueError, match=match):
            wb.kv_attend_chunk(**{**good, **kw})
    with pytest.raises(Exception, match="kv_attend_chunk"):                          # q of another type than the cache
        wb.kv_attend_chunk(**{**good, "q": q.half(), "o": o.half()})
    with pytest.raises(Exception, match="kv_attend_chunk"):                          # in place
        wb.kv_attend_chunk(**{**good, "o": q})

    x, at, freqs = cu(3, 4, 64), cu(3, dtype=i), cu(32, dtype=f64)
    good = dict(q=x, k=x.clone(), positions=at, freqs=freqs)
    for match, kw in [("q: expected", dict(q=x[0])), ("q: expected", dict(q=x.to(f8))), ("q: expected", dict(q=cu(3, 4, 128)[..., ::2])),
                      ("freqs: expected", dict(freqs=freqs.float())), ("freqs: expected", dict(freqs=freqs.view(1, 32))),
                      ("freqs: 33 pairs", dict(freqs=cu(33, dtype=f64))), ("freqs: expected", dict(freqs=host(freqs))),
                      ("positions: expected", dict(positions=at.float())), ("positions: expected", dict(positions=cu(4, dtype=i))),
                      ("positions: expected", dict(positions=cu(6, dtype=long)[::2])), ("q_weight: expected", dict(q_weight=cu(32))),
                      ("q_weight: expected", dict(q_weight=cu(64, dtype=f32))), ("k_weight: expected", dict(k_weight=cu(1, 64))),
                      ("k: expected", dict(k=cu(2, 4, 64))), ("k: expected", dict(k=cu(3, 4, 32))), ("k: expected", dict(k=x.float())),
                      ("k: expected", dict(k=x[0])), ("q_out: expected", dict(q_out=cu(3, 5, 64))), ("k_out: expected", dict(k_out=x.float())),
                      ("q_out: expected", dict(q_out=cu(3, 4, 128)[..., ::2])), ("q_out: expected", dict(q_out=x[0]))]:
        with pytest.raises(ValueError, match=match):
            wb.qk_rotate(**{**good, **kw})
    for kw in (dict(q_out=cu(1, 1, 64).expand(3, 4, 64)), dict(k=x), dict(eps=-1.0), dict(magnitude=math.nan)):
        with pytest.raises(Exception, match="qk_rotate"):
            wb.qk_rotate(**{**good, **kw})

    x, tok, lp = cu(3, 50), cu(3, dtype=long), cu(3, dtype=f32)
    ids, top = cu(3, 4, dtype=i), cu(3, 4, dtype=f32)
    good = dict(logits=x, tokens=tok, logprob=lp)
    for match, kw in [("logits: expected", dict(logits=x[0])), ("logits: expected", dict(logits=x.to(f8))), ("logits: expected", dict(logits=cu(3, 100)[:, ::2])),
                      ("tokens: expected", dict(tokens=tok.float())), ("tokens: expected", dict(tokens=cu(4, dtype=long))), ("logprob: expected", dict(logprob=cu(3))),
                      ("logprob: expected", dict(logprob=cu(2, dtype=f32))), ("entropy: expected", dict(entropy=cu(3))),
                      ("both or neither", dict(top_ids=ids)), ("both or neither", dict(top_logprobs=top)), ("top_ids: expected", dict(top_ids=tok, top_logprobs=top)),
                      ("top_ids: expected", dict(top_ids=ids.long(), top_logprobs=top)), ("top_logprobs: expected", dict(top_ids=ids, top_logprobs=top[:, :3])),
                      ("logprob: expected", dict(logprob=host(lp)))]:
        with pytest.raises(ValueError, match=match):
            wb.token_logprobs(**{**good, **kw})
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=1e-40), dict(top_ids=cu(3, 51, dtype=i), top_logprobs=cu(3, 51, dtype=f32))):
        with pytest.raises(Exception, match="token_logprobs"):
            wb.token_logprobs(**{**good, **kw})
    torch.cuda.synchronize()
    assert (o == 0).all() and (lp == 0).all()


@pytest.mark.parametrize("R", [65, 4097, 65536])
def test_many_requests_some_without_new_tokens(R):
    """As many requests as there may be, two of three without a new token; each row sees one token, whose value it has."""
    import linear_attn_decode_amd as wb
    g = torch.Generator().manual_seed(R)
    k, v = (rand(g, 5, 2, 8, 64, dtype="f16").cuda() for _ in range(2))
    new = (torch.rand(R, generator=g) < 0.34).int()
    new[-1] = 0
    starts = torch.cat([torch.zeros(1, dtype=torch.int32), new.cumsum(0).int()])
    N = int(starts[-1])
    q = rand(g, N + 3, 2, 64, dtype="f16").cuda()
    o, lse = torch.full_like(q, 7.0), torch.full((N + 3, 2), 7.0, device="cuda")
    table = (torch.arange(R, dtype=torch.int32) % 5).view(R, 1)
    wb.kv_attend_chunk(q, k, v, table.cuda(), torch.ones(R, dtype=torch.int32, device="cuda"), starts.cuda(), o, lse=lse)
    torch.cuda.synchronize()
    page = table[new.bool(), 0].long().cuda()
    assert torch.equal(o[:N], v[page, :, 0]) and (o[N:] == 7).all() and (lse[N:] == 7).all()


@pytest.mark.parametrize("K", [0, 1, 32, 33, 64])
def test_largest_vocabulary(K):
    """2^24 columns (8 fewer with more than 32 alternatives, from any alignment on); the same with every column equal, where
    no group of columns can be left out."""
    import linear_attn_decode_amd as wb
    V = 2 ** 24
    x = torch.randn((1, V), generator=torch.Generator().manual_seed(K)).bfloat16().cuda()
    if K > 32:
        with pytest.raises(RuntimeError, match="EUNSUPPORTED"):
            wb.token_logprobs(x, torch.tensor([0]).cuda(), torch.empty(1, device="cuda"), top_logprobs=torch.empty((1, K), device="cuda"),
                              top_ids=torch.empty((1, K), dtype=torch.int32, device="cuda"))
        x = x[:, 7:V - 1]
    check_logprobs(x, [x.shape[1] - 1], K)
    if K > 32:
        x.fill_(2.5)
        check_logprobs(x, [12345], K)
