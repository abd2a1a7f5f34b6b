"""fuse_attend_chunks on the GPU against its fp64 statement: every storage,
layout, type and head layout, ragged and empty chunks, selections that leave a
request's chunks without a key, several new tokens, and what must not reach a
row (selected tokens, unused pages and rows, later tokens)."""

import numpy as np
import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

from cache_ops import DT, KIND, Attend, AttendCase, f64

pytestmark = pytest.mark.gpu


def check(a: Attend, O=None):
    O = a.run() if O is None else O
    fk.check_errors(a.ws)
    want, tol = a.reference()
    err = np.abs(f64(O) - want)
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(err / tol)), np.argwhere(bad)[:3].tolist())


RAGGED = dict(lens=[[33, 1, 64], [7], [16, 0, 129, 31]], n_query=[5, 9, 17], k=[13, 0, 60])


@pytest.mark.parametrize("storage", ["u4", "u8", "bf16"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 8, 128), (16, 2, 64), (6, 3, 128)])
def test_bf16_layers(storage, paged, heads):
    check(Attend(AttendCase(**RAGGED, storage=storage, paged=paged, heads=heads, gap=3)))


@pytest.mark.parametrize("storage", ["u4", "u8", "f32"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128)])
def test_fp32_layers(storage, paged, heads):
    check(Attend(AttendCase(**RAGGED, storage=storage, paged=paged, heads=heads, dtype="f32", base=1e4)))


@pytest.mark.parametrize("new", [2, 3, 8])
@pytest.mark.parametrize("dtype,storage,heads", [("bf16", "u4", (8, 1, 128)), ("bf16", "u8", (4, 4, 64)),
                                                 ("bf16", "bf16", (8, 2, 128)), ("f32", "u4", (4, 1, 64))])
def test_several_new_tokens(new, dtype, storage, heads):
    check(Attend(AttendCase(**{**RAGGED, "n_query": [new, 9, 17]}, storage=storage, dtype=dtype,
                            heads=heads, new=new, paged=True, block_size=24, gap=1)))


@pytest.mark.parametrize("storage", ["u4", "bf16"])
def test_requests_without_context_or_with_everything_selected(storage):
    lens = [[], [40, 25], [0], [1]]
    check(Attend(AttendCase(lens=lens, n_query=[1, 1, 2, 1], k=[0, 65, 0, 1], storage=storage)))


@pytest.mark.parametrize("block_size", [1, 5, 16, 24, 128])
def test_pages_that_end_inside_a_segment(block_size):
    check(Attend(AttendCase(lens=[[100, 37]], n_query=[3], k=[20], paged=True, block_size=block_size,
                            heads=(4, 2, 128))))


def test_far_positions():
    # angles of positions near 2^23 keep their accuracy
    check(Attend(AttendCase(lens=[[50, 70]], n_query=[2], k=[9], pos_shift=(1 << 23) + 12345,
                            dtype="f32", heads=(4, 2, 64), base=1e4)))


@pytest.mark.parametrize("storage", ["u4", "u8", "bf16"])
def test_longer_contexts(storage):
    # several segments per chunk, several requests a wave
    check(Attend(AttendCase(lens=[[700, 513, 900], [1025]], n_query=[40, 3], k=[300, 100],
                            storage=storage, heads=(8, 2, 128))))


def test_many_requests_and_chunks():
    # more than one launch's tables of requests and of chunks
    n = 530
    check(Attend(AttendCase(lens=[[3, 2, 4, 1]] * n, n_query=[1 + i % 3 for i in range(n)],
                            k=[i % 5 for i in range(n)], heads=(2, 1, 64))))


def test_more_chunks_than_a_join_holds_at_once():
    check(Attend(AttendCase(lens=[[2, 1, 3] * 200, [5]], n_query=[3, 1], k=[100, 0], heads=(4, 2, 128), new=1)))


def test_constant_values_and_keys():
    # groups with scale 0, as a KIVI constant group stores them
    a = Attend(AttendCase(lens=[[48]], n_query=[2], k=[0], heads=(4, 2, 128)))
    a.vs.zero_()
    a.ks[:, 0].zero_()
    a.keys = [np.where(np.arange(2)[:, None] == 0, f64(a.kz)[0], a.keys[0])]
    a.vals = [np.broadcast_to(f64(a.vz)[..., None], a.vals[0].shape)]
    check(a)


@pytest.mark.parametrize("storage", ["u4", "bf16"])
@pytest.mark.parametrize("paged", [False, True])
def test_selected_tokens_do_not_reach_a_row(storage, paged):
    a = Attend(AttendCase(lens=[[60, 45]], n_query=[4], k=[30], storage=storage, paged=paged,
                          heads=(4, 2, 128)))
    bs, flat = 16, [60, 45]
    for p in a.idx_list[0]:
        i, t = (0, p) if p < 60 else (1, p - 60)
        at = (int(a.tables[i][t // bs]), t % bs) if paged else (int(p),)
        if storage == "bf16":
            a.K[at], a.V[at] = float("nan"), float("inf")
        else:
            a.vs[at], a.vz[at] = float("nan"), float("inf")
    check(a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_later_tokens_do_not_reach_a_row(dtype):
    c = AttendCase(lens=[[40]], n_query=[9], k=[5], new=4, dtype=dtype, heads=(4, 2, 64))
    a = Attend(c)
    want, tol = a.reference()
    n = 5 + 9
    a.Vs[n - 2:n] = float("nan")                         # values of the last two new tokens
    a.Ks[n - 1] = float("inf")
    got = f64(a.run())
    assert (np.abs(got[:2] - want[:2]) <= tol[:2]).all()
    assert np.isnan(got[2:]).all()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_what_is_seen_does_reach_a_row(value):
    a = Attend(AttendCase(lens=[[40]], n_query=[2], k=[0], storage="bf16", heads=(4, 2, 128)))
    a.V[7, 0, 3] = value
    got = f64(a.run())
    assert not np.isfinite(got[0, :2, 3]).any() and np.isfinite(got[0, 2:]).all()
    assert np.isfinite(np.delete(got[0, :2], 3, -1)).all()


@pytest.mark.parametrize("storage", ["u4", "bf16"])
def test_block_ids_outside_the_pool_are_dropped_and_reported(storage):
    a = Attend(AttendCase(lens=[[40, 20]], n_query=[2], k=[0], paged=True, storage=storage,
                          heads=(4, 2, 128)))
    a.tables[0][1] = a.n_blocks + 5
    a.tables[1][0] = -3
    a.run()
    with pytest.raises(fk.FuseError) as e:
        fk.check_errors(a.ws)
    assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
    want = Attend.__new__(Attend)
    want.__dict__.update(a.__dict__)
    gone = np.r_[16:32, 40:56]
    want.idx_list = [gone]                                # as if selected, with no refreshed row
    O, tol = want.reference()
    assert (np.abs(f64(a.O) - O) <= tol).all()
    a.run()                                               # the error word was cleared, the call repeats
    with pytest.raises(fk.FuseError):
        fk.check_errors(a.ws)


def test_unordered_or_outside_selection_is_reported():
    for bad in ([5, 5, 9], [9, 4, 20], [3, 8, 40], [-1, 2, 3]):
        a = Attend(AttendCase(lens=[[40]], n_query=[2], k=[3], heads=(4, 2, 64)))
        a.idx.copy_(torch.tensor(bad, dtype=torch.int32))
        a.run()
        with pytest.raises(fk.FuseError) as e:
            fk.check_errors(a.ws)
        assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS


def test_cache_past_four_gigabytes():
    # pages whose byte offsets pass 2^32 and whose element offsets pass 2^31
    check(Attend(AttendCase(lens=[[70, 33]], n_query=[2], k=[10], storage="bf16", paged=True,
                            heads=(8, 8, 128), spare_blocks=140000)))


def test_repeated_runs_are_equal_bit_for_bit_and_other_memory_is_left():
    a = Attend(AttendCase(**RAGGED, gap=2))
    one = a.run().clone()
    a.O.zero_()
    a.ws[256:].fill_(0xA5)                               # scratch is written before it is read
    assert torch.equal(a.run(), one)


def test_other_stream_and_graph():
    a = Attend(AttendCase(**RAGGED, paged=True))
    want = a.run().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.O.zero_()
    torch.cuda.synchronize()
    a.run(stream=s)
    s.synchronize()
    assert torch.equal(a.O, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        a.run(stream=s)
    for seed in (1, 2):
        q = torch.randn(a.Q.shape, generator=torch.Generator().manual_seed(seed)).to(a.Q.dtype)
        a.Q.copy_(q)
        g.replay()
        got = a.O.clone()
        assert torch.equal(a.run(), got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_requests_of_one_token_follow_what_writes_their_rows(dtype):
    """Requests of a single token without context leave nothing but the join,
    which must not read its rows before the kernel that writes them (a prompt
    attention) has ended."""
    T, H, d = 2048, 8, 128
    g = torch.Generator().manual_seed(11)
    Q, K, V = (torch.randn(T, H, d, generator=g).to(DT[dtype]).cuda() for _ in range(3))
    desc = fk.layer_desc(64, H, H, d, 1e6, KIND[dtype])
    prompt = fk.RequestTable([fk.Request(0, 0, 0, 0, T, 0, 0, 0)])
    reqs = fk.RequestTable([fk.Request(i, 0, 0, i, 0, 1, 0, 0) for i in range(T)])
    none = fk.ChunkTable([], fk.FUSE_KV_CONTIGUOUS, fk.FUSE_U4_ASYM)
    ws, ws2 = fk.alloc_workspace(desc, prompt), fk.alloc_attend_workspace(desc, none, reqs, 1)
    P, O = torch.zeros_like(Q), torch.zeros_like(Q)
    for _ in range(3):
        P.zero_()
        fk.attend_prompt(desc, prompt, Q, K, V, P, ws)
        fk.attend_chunks(desc, none, reqs, 1, Q, None, K, P, O, ws2)
        # one key: its weight is 1 and the row its value
        assert torch.equal(O, P) and bool((P != 0).any(-1).all())
    fk.check_errors(ws2)


WHERE = ["chunk", "side", "own"]             # of a key: a cached chunk, an earlier query token, the token itself


@pytest.mark.parametrize("dtype,heads", [("bf16", (4, 2, 128)), ("bf16", (8, 1, 64)), ("f32", (4, 2, 64))])
@pytest.mark.parametrize("where", WHERE)
def test_a_key_of_score_minus_infinity_has_no_weight(dtype, heads, where):
    a = Attend(AttendCase(lens=[[40, 30]], n_query=[3], k=[0], storage=dtype, dtype=dtype, heads=heads))
    a.Q[..., 0] = 1.0
    if where == "chunk":
        a.idx_list = [np.array([7])]
    want, tol = a.reference(unseen={"chunk": [], "side": [0], "own": [2]}[where])
    rows, i = {"chunk": (a.K, 7), "side": (a.Ks, 0), "own": (a.Ks, 2)}[where]
    rows[i, :, 0] = -float("inf")
    got = f64(a.run())
    fk.check_errors(a.ws)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("dtype,heads", [("bf16", (4, 2, 128)), ("bf16", (8, 1, 64)), ("f32", (4, 2, 64))])
@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_an_infinite_value_gives_infinity(dtype, heads, where, value):
    a = Attend(AttendCase(lens=[[40, 30]], n_query=[3], k=[0], storage=dtype, dtype=dtype, heads=heads))
    want, tol = a.reference()
    rows, i = {"chunk": (a.V, 7), "side": (a.Vs, 0), "own": (a.Vs, 2)}[where]
    rows[i, 0, 3] = value
    got = f64(a.run())
    g = heads[0] // heads[1]
    assert (got[:, :g, 3] == value).all()
    got[:, :g, 3] = want[:, :g, 3]
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_infinite_value_of_the_only_key(dtype):
    # its weight is 1, which 16 bits hold without a remainder
    a = Attend(AttendCase(lens=[[1]], n_query=[1], k=[0], storage=dtype, dtype=dtype, heads=(4, 2, 128)))
    a.Ks[0].zero_()
    a.Q.zero_()
    want, tol = a.reference()
    a.V[0, 1, 5] = float("inf")
    got = f64(a.run())
    assert (got[:, 2:, 5] == np.inf).all()
    got[:, 2:, 5] = want[:, 2:, 5]
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("storage", ["u4", "u8"])
def test_an_infinite_key_scale(storage, dtype):
    # every key of the first chunk scores -infinity; the second one is left
    a = Attend(AttendCase(lens=[[30, 40]], n_query=[3], k=[0], storage=storage, dtype=dtype, heads=(4, 2, 128)))
    a.Q[..., 5] = -1.0
    a.idx_list = [np.arange(30)]
    want, tol = a.reference()
    a.ks[0, :, 5] = float("inf")
    a.K[:30, :, 2 if storage == "u4" else 5] |= 0x10     # no code of channel 5 is 0
    got = f64(a.run())
    fk.check_errors(a.ws)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("storage", ["u4", "u8"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("paged", [False, True])
def test_scales_of_a_wholly_selected_chunk_do_not_reach_a_row(storage, dtype, value, paged):
    a = Attend(AttendCase(lens=[[70, 45]], n_query=[4], k=[70], storage=storage, dtype=dtype, paged=paged,
                          heads=(4, 2, 128)))
    a.idx_list = [np.arange(70)]
    a.idx.copy_(torch.arange(70, dtype=torch.int32))
    a.ks[0], a.kz[0] = value, value
    check(a)


def test_a_request_table_that_grows_in_place():
    """A decode loop raises n_query of the host table's last request by one a
    step: each step's rows are those of tables built anew."""
    c = AttendCase(lens=[[70, 33], [50]], n_query=[2, 4], k=[9, 0], heads=(4, 2, 128), gap=5)
    a = Attend(c)
    room = [torch.full_like(x, float("nan")) for x in (a.Ks, a.Vs)]
    for x, y in zip(room, (a.Ks, a.Vs)):
        x.normal_(generator=torch.Generator("cuda").manual_seed(3))
        x[~torch.isnan(y)] = y[~torch.isnan(y)]
    a.Ks, a.Vs = room
    for step in range(5):
        if step:
            a.reqs.host[1].n_query += 1
        a.ws = fk.alloc_attend_workspace(a.desc, a.chunks, a.reqs, 1)
        got = a.run().clone()
        fresh = fk.RequestTable([fk.Request(r.row0, r.score0, r.sel0, r.out0, r.n_ctx, r.n_query, r.k, 0)
                                 for r in a.reqs.host[:a.reqs.n]])
        want = torch.zeros_like(got)
        fk.attend_chunks(a.desc, a.chunks, fresh, 1, a.Q, a.idx, a.Ks, a.Vs, want, a.ws)
        fk.check_errors(a.ws)
        assert torch.equal(got, want), step


def test_a_request_table_edited_in_place_on_another_stream_and_before_a_capture():
    c = AttendCase(lens=[[40]], n_query=[4], k=[3], heads=(4, 2, 64))
    a = Attend(c)
    s = torch.cuda.Stream()
    a.reqs.host[0].n_query = 3                           # the last row is dropped again
    torch.cuda.synchronize()
    a.run(stream=s)
    s.synchronize()
    got, want = a.O.clone(), torch.zeros_like(a.O)
    fresh = fk.RequestTable([fk.Request(0, 0, 0, 0, 40, 3, 3, 0)])
    fk.attend_chunks(a.desc, a.chunks, fresh, 1, a.Q, a.idx, a.Ks, a.Vs, want, a.ws)
    assert torch.equal(got, want)
    a.reqs.host[0].n_query = 2
    g = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError):
        with torch.cuda.graph(g, stream=s):
            a.run(stream=s)
    a.reqs.update()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        a.run(stream=s)
    g.replay()
    got = a.O.clone()
    assert torch.equal(a.run(stream=s.cuda_stream), got) and not torch.equal(got, want)
    fk.check_errors(a.ws)


SLOT = {"u4": 64, "u8": 32, "bf16": 16, "f32": 32}       # keys that an item takes at a time


def check_long(a: Attend, at_least):
    """A call whose items hold at_least keys on average, at six rows and heads
    (a key's weight, scales and position show in each)."""
    Hq, new = a.c.heads[0], a.c.new
    n = sum(a.n_ctx) + sum(r.k + r.n_query - new for r in a.reqs.host[:a.reqs.n])
    assert n / a.segments() >= at_least > SLOT[a.c.storage]
    got = f64(a.run())
    fk.check_errors(a.ws)
    rows = [(u, h) for u in (0, len(got) - 1) for h in (0, Hq // 3, Hq - 1)]
    want, tol = a.reference(rows)
    for i in rows:
        err = np.abs(got[i] - want[i])
        assert (err <= tol[i]).all(), (i, float(np.nanmax(err / tol[i])))


@pytest.mark.parametrize("score,value", [(6.0, 0.0), (0.0, 10.0), (6.0, 10.0)])
@pytest.mark.parametrize("dtype,storage,paged,d", [
    ("bf16", "u4", False, 128), ("bf16", "u4", True, 128), ("bf16", "u4", True, 64), ("bf16", "u8", False, 128),
    ("bf16", "u8", True, 64), ("bf16", "bf16", False, 64), ("bf16", "bf16", True, 128), ("f32", "u4", False, 64),
    ("f32", "u8", True, 128), ("f32", "f32", False, 128)])
def test_items_of_several_slots(dtype, storage, paged, d, score, value):
    # 256 keys an item; from slot to slot the scores rise by 6 (8.7 in log2: past
    # what the running maximum may lag) or stay, the values' scales by 2^10 over
    # an item; the selection hides every third key or so
    steps = 256 // SLOT[storage]
    a = Attend(AttendCase(lens=[[30000, 27000]], n_query=[9], k=[18000], dtype=dtype, storage=storage, paged=paged,
                          block_size=24, heads=(8, 1, d), new=8, rise=(SLOT[storage], steps, score, value / (steps - 1))))
    check_long(a, 160)


@pytest.mark.parametrize("dtype,storage,paged", [("bf16", "u4", True), ("bf16", "u8", False), ("bf16", "bf16", False),
                                                 ("f32", "u4", False)])
def test_items_of_1024_keys(dtype, storage, paged):
    steps = 1024 // SLOT[storage]
    a = Attend(AttendCase(lens=[[120000, 105000]], n_query=[9], k=[500], dtype=dtype, storage=storage, paged=paged,
                          block_size=1000, heads=(8, 1, 64), new=8, rise=(SLOT[storage], steps, 6.0, 10.0 / steps)))
    check_long(a, 850)                                   # fp32 items: 992, in whole steps of 32


@pytest.mark.parametrize("dtype,storage", [("bf16", "u4"), ("bf16", "bf16"), ("f32", "u8")])
@pytest.mark.parametrize("heads,new", [((4, 2, 64), 1), ((3, 3, 64), 2), ((8, 1, 128), 3)])
def test_long_chunks_beside_short_ones(dtype, storage, heads, new):
    # chunks of very different lengths, empty ones, requests without any, long
    # and short generations; segments that do and do not fill a CTA
    lens = [[5] * 40 + [1500, 0, 0, 3], [], [1, 0, 700], [0], [2] * 300 + [900] + [1] * 300]
    check(Attend(AttendCase(lens=lens, n_query=[3, 300, 7, 4, 9], k=[100, 0, 1, 0, 400], dtype=dtype, storage=storage,
                            heads=heads, new=new)))


def test_one_long_generation_among_many_requests():
    # more requests than a launch takes the side rows of, most with none
    n = 600
    q = [1 + (i % 7 == 0) * (i % 40) for i in range(n)]
    q[333] = 2000
    check(Attend(AttendCase(lens=[[3] if i % 3 else [] for i in range(n)], n_query=q, k=[0] * n, heads=(2, 1, 64))))


def test_more_segments_than_a_launch_takes():
    """515 chunks of 132 segments each: past the 65535 that a launch counts.
    Every page of every chunk is the same one, so the sum over its keys counts
    n times.  Fp32 sums: 1024 keys an item, then the items one by one."""
    Hq, d, bs, pages, per_req, n_req = 8, 64, 1024, 132, 103, 5
    g = torch.Generator().manual_seed(2)
    mk = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    K, V = mk(1, bs, 1, d), mk(1, bs, 1, d)
    Q, Ks, Vs = 1.5 * mk(n_req, Hq, d), mk(n_req, 1, d), mk(n_req, 1, d)
    table = torch.zeros(pages, dtype=torch.int32, device="cuda")
    n_ctx = per_req * pages * bs
    reqs = fk.RequestTable([fk.Request(i * (n_ctx + 1), 0, 0, i, n_ctx, 1, 0, 0) for i in range(n_req)])
    entries = []
    for c in range(n_req * per_req):
        e = fk.Chunk()
        e.k, e.v, e.block_table = K.data_ptr(), V.data_ptr(), table.data_ptr()
        e.dst_row, e.pos, e.len = c // per_req * (n_ctx + 1) + c % per_req * pages * bs, 0, pages * bs
        entries.append(e)
    chunks = fk.ChunkTable(entries, fk.FUSE_KV_PAGED, fk.FUSE_BF16, block_size=bs, n_pool_blocks=1, keep=[K, V, table])
    desc = fk.layer_desc(64, Hq, 1, d, 1e6, fk.FUSE_BF16)
    ws, O = fk.alloc_attend_workspace(desc, chunks, reqs, 1), torch.zeros_like(Q)
    assert (ws.numel() - 256) // (8 * (8 + 4 * d)) == n_req * per_req * pages
    fk.attend_chunks(desc, chunks, reqs, 1, Q, None, Ks, Vs, O, ws)
    fk.check_errors(ws)
    k, v, n = f64(K)[0, :, 0], f64(V)[0, :, 0], per_req * pages
    for r in range(n_req):
        for h in range(Hq):
            q = f64(Q)[r, h] / np.sqrt(d)
            s, s1 = k @ q, f64(Ks)[r, 0] @ q
            m = max(s.max(), s1)
            w, w1 = n * np.exp(s - m), np.exp(s1 - m)
            l = w.sum() + w1
            want, A = (w @ v + w1 * f64(Vs)[r, 0]) / l, (w @ np.abs(v) + w1 * np.abs(f64(Vs)[r, 0])) / l
            S = max((np.abs(k) @ np.abs(q)).max(), np.abs(f64(Ks)[r, 0]) @ np.abs(q))
            e = S * ((d + 16) * 2.0 ** -23 + 2.0 ** -20)
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * e + (bs + n) * 2.0 ** -24) * A
            assert (np.abs(f64(O)[r, h] - want) <= tol).all(), (r, h)
