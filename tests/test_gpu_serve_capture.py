"""Captured serving calls (include/wbserve.h) in the forms that take two launches: what the first
leaves in the workspace is read by the second, and replays go with other lengths. Every replay
gives the eager call's bits."""
import numpy as np
import pytest

from oracle import serving as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# (the last joins in one launch)
@pytest.mark.parametrize("kv,D,H,G,R,width", [("bf16", 256, 2, 8, 4, 600), ("bf16", 256, 2, 8, 40, 60), ("f16", 256, 2, 8, 70, 60),
                                              ("e4m3", 128, 4, 8, 100, 40), ("bf16", 128, 8, 4, 6, 200)])
def test_captured_attention_replays_with_other_lengths(kv, D, H, G, R, width):
    import linear_attn_decode_amd as wb
    print(f"[case] captured attend kv={kv} D={D} H={H} G={G} R={R}", flush=True)
    g = torch.Generator().manual_seed(R)
    rng = np.random.default_rng(R)
    page, pages = 16, 700
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[kv]
    k, v = (torch.randn((pages, H, page, D), generator=g).to(dt).cuda() for _ in range(2))
    ks, vs = (torch.rand((pages, H, page), generator=g).cuda() if kv == "e4m3" else None for _ in range(2))
    table = torch.from_numpy(rng.integers(0, pages, (R, width)).astype(np.int32)).cuda()
    q = torch.randn((R, H * G, D), generator=g).to(torch.bfloat16 if kv == "e4m3" else dt).cuda()
    lens = torch.ones(R, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((R, H * G), device="cuda")
    o_want, lse_want = torch.empty_like(o), torch.empty_like(lse)
    call = lambda o, lse: wb.kv_attend(q, k, v, table, lens, o, lse=lse, k_scale=ks, v_scale=vs)
    call(o_want, lse_want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o, lse)
        call(o, lse)                                     # (in the first one's workspace, perhaps)
    most = width * page
    for step in range(8):
        n = [np.full(R, most), np.zeros(R), rng.integers(0, most + 1, R), np.where(np.arange(R) == R - 1, most, 1),
             np.where(np.arange(R) == 0, most, 0), rng.integers(0, 300, R), rng.integers(0, most + 1, R), np.full(R, most)][step]
        lens.copy_(torch.from_numpy(n.astype(np.int32)))
        o.fill_(7)
        lse.fill_(7)
        call(o_want, lse_want)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o_want) and torch.equal(lse, lse_want), step
        assert torch.isneginf(lse).all(1).cpu().tolist() == (n == 0).tolist()
        q.copy_(torch.randn(q.shape, generator=g).to(q.dtype))


@pytest.mark.parametrize("R,n_slots", [(300, 9000), (1500, 3000)])
def test_captured_plan_in_place_replays(R, n_slots):
    """In place and of many slots or requests: the sums in one launch, the slots in another."""
    import linear_attn_decode_amd as wb
    print(f"[case] captured plan R={R} n_slots={n_slots}", flush=True)
    rng = np.random.default_rng(R)
    page, width, pages = 16, 40, 60000
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()
    host_table, host_free = np.full((R, width), -1, np.int32), rng.permutation(pages).astype(np.int32)
    lens, more, table, free, n_free = i32([0] * R), i32([0] * R), i32(host_table), i32(host_free), i32([pages])
    slots, starts, status = torch.empty(n_slots, dtype=torch.int64, device="cuda"), i32([0] * (R + 1)), i32([9])
    call = lambda: wb.plan_pages(lens, more, table, free, n_free, page, slots, starts, status)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    n, left = np.zeros(R, np.int32), pages
    for step in range(7):
        m = rng.integers(0, 2 * n_slots // R, R) * (rng.random(R) < 0.6)
        m[rng.integers(0, R)] += 1
        if step == 3:
            m[0] += n_slots                              # more than there are slots, or than a table holds: nothing changes
        want = O.plan(n, m, host_table, host_free, left, page, n_slots)
        more.copy_(torch.from_numpy(m.astype(np.int32)))
        slots.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        for name, a, b in zip(("table", "slots", "starts", "lens", "n_free", "status"), (table, slots, starts, lens, n_free, status), want):
            assert np.array_equal(a.cpu().numpy().reshape(np.shape(b)), b), (name, step)
        assert (want[5] != 0) == (step == 3)
        host_table, n, left = want[0], want[3].astype(np.int32), int(want[4])
