"""Page upkeep on the GPU against lists in Python: fork, free, compact and
copy, their refusals on the device, and a run of the cache operators together."""

import numpy as np
import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

import cache_ops
from cache_ops import (Attend, AttendCase, compact_reference, f64, fork_reference, page_table)

pytestmark = pytest.mark.gpu


def draw(seed, n_blocks, n_seq, max_len, bs, share=True):
    """Random tables over a pool: (tables, lens, refs); some sequences share pages."""
    rng = np.random.default_rng(seed)
    perm, at = rng.permutation(n_blocks), 0
    tables, lens = [], []
    for i in range(n_seq):
        n = int(rng.integers(0, max_len + 1))
        nb = -(-n // bs)
        if at + nb > n_blocks:
            break
        tables.append(perm[at:at + nb].astype(np.int32))
        lens.append(n)
        at += nb
    if share and len(tables) > 2:
        tables.append(tables[1].copy())
        lens.append(lens[1])
    refs = np.zeros(n_blocks, np.int32)
    for t in tables:
        np.add.at(refs, t, 1)
    return tables, lens, refs


def dev(tables):
    return [torch.from_numpy(np.ascontiguousarray(t, dtype=np.int32)).cuda() for t in tables]


def lists(tables):
    return [t.cpu().tolist() for t in tables]


def moves_of(m):
    m = m.cpu().tolist()
    return [(m[2 + 2 * i], m[3 + 2 * i]) for i in range(m[0])], m[1]


@pytest.mark.parametrize("seed,n_blocks,n_seq,max_len,bs,fan", [
    (0, 64, 4, 100, 16, 1), (1, 301, 20, 150, 16, 3), (2, 5000, 60, 900, 24, 2),
    (3, 33001, 1100, 40, 1, 2), (4, 1, 1, 0, 16, 1), (5, 40007, 7, 3000, 7, 5)])
def test_fork_then_drop(seed, n_blocks, n_seq, max_len, bs, fan):
    tables, lens, refs = draw(seed, n_blocks, n_seq, max_len, bs)
    want = fork_reference(tables * fan, lens * fan, refs, bs)
    if want is None:
        pytest.skip("the draw leaves too few free pages")
    d_src = dev(tables)
    d_dst = [torch.full((max(1, -(-n // bs)),), -9, dtype=torch.int32, device="cuda") for n in lens * fan]
    d_refs = torch.from_numpy(refs).cuda()
    src = page_table(d_src * fan, lens * fan, bs, n_blocks)
    dst = page_table(d_dst, lens * fan, bs, n_blocks)
    moves, ws = fk.alloc_moves(len(lens) * fan + 3), fk.alloc_pages_workspace(src)
    moves[2:] = -5
    fk.pages_fork(src, dst, d_refs, moves, ws)
    fk.check_errors(ws)
    assert [t[:-(-n // bs)] for t, n in zip(lists(d_dst), lens * fan)] == want[0]
    assert d_refs.cpu().tolist() == want[1]
    got, live = moves_of(moves)
    assert got == want[2] and live == sum(r > 0 for r in want[1])
    assert (moves[2 + 2 * len(got):] == -5).all()
    assert lists(d_src) == [t.tolist() for t in tables]
    fk.pages_free(dst, d_refs, ws)
    fk.check_errors(ws)
    assert d_refs.cpu().tolist() == refs.tolist()


@pytest.mark.parametrize("seed,n_blocks,n_seq,max_len,bs", [
    (0, 64, 4, 100, 16), (1, 301, 20, 150, 16), (2, 5000, 60, 900, 24), (3, 33001, 1100, 20, 1),
    (4, 1, 1, 0, 16), (5, 40007, 7, 3000, 7), (6, 257, 40, 64, 4), (7, 96, 200, 16, 16)])
def test_compact(seed, n_blocks, n_seq, max_len, bs):
    tables, lens, refs = draw(seed, n_blocks, n_seq, max_len, bs)
    want = compact_reference(tables, refs)
    d_tab, d_refs = dev(tables), torch.from_numpy(refs).cuda()
    d_refs0 = d_refs
    # the first table is given twice: rewritten once
    tab = page_table(d_tab + d_tab[:1], lens + lens[:1], bs, n_blocks)
    moves, ws = fk.alloc_moves(n_blocks // 2), fk.alloc_pages_workspace(tab)
    fk.pages_compact(tab, d_refs, moves, ws)
    fk.check_errors(ws)
    assert lists(d_tab) == want[0] and d_refs0.cpu().tolist() == want[1]
    got, live = moves_of(moves)
    assert got == want[2] and live == want[3]
    fk.pages_compact(tab, d_refs, moves, ws)                 # packed: nothing moves
    fk.check_errors(ws)
    assert moves_of(moves) == ([], want[3]) and lists(d_tab) == want[0]


@pytest.mark.parametrize("storage", ["u4", "u8", "bf16", "f32"])
@pytest.mark.parametrize("heads,bs,layers", [((2, 64), 16, 1), ((8, 128), 16, 3), ((3, 128), 5, 2), ((1, 64), 1, 70)])
def test_copy(storage, heads, bs, layers):
    Hkv, d = heads
    nb = 40
    g = torch.Generator().manual_seed(1)
    code = storage in ("u4", "u8")
    per = d // 2 if storage == "u4" else d

    def pool():
        if code:
            return torch.randint(0, 256, (nb, bs, Hkv, per), generator=g, dtype=torch.uint8).cuda()
        return torch.randn(nb, bs, Hkv, d, generator=g).to(cache_ops.DT[storage]).cuda()
    k, v = [pool() for _ in range(layers)], [pool() for _ in range(layers)]
    sc = [torch.randn(nb, bs, Hkv, generator=g).half().cuda() for _ in range(2 * layers)] if code else []
    pools = fk.PagePools(k, v, cache_ops.KIND[storage], bs, sc[:layers], sc[layers:])
    perm = torch.randperm(nb, generator=g).int()
    pairs = [(int(perm[i]), int(perm[20 + i])) for i in range(17)] + [(int(perm[0]), int(perm[39]))]
    moves, ws = fk.alloc_moves(25), fk.alloc_pages_workspace(None)
    moves[0] = len(pairs)
    moves[2:2 + 2 * len(pairs)] = torch.tensor(pairs, dtype=torch.int32).reshape(-1).cuda()
    before = [x.clone() for x in k + v + sc]
    desc = fk.layer_desc(64, Hkv, Hkv, d, 1e4, fk.FUSE_BF16)
    fk.pages_copy(desc, pools, moves, ws)
    fk.check_errors(ws)
    for x, y in zip(k + v + sc, before):
        for a, b in pairs:
            y[b] = y[a]
        assert torch.equal(x.view(torch.uint8) if not code else x, y.view(torch.uint8) if not code else y)


def test_copy_past_four_gigabytes():
    Hkv, d, bs, nb = 8, 128, 16, 140001
    k = torch.empty(nb, bs, Hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(nb, bs, Hkv, d, dtype=torch.bfloat16, device="cuda")
    for i, x in enumerate((k, v)):
        x[0], x[nb - 1], x[nb - 2] = 1 + i, 3 + i, 5 + i
    desc = fk.layer_desc(64, Hkv, Hkv, d, 1e4, fk.FUSE_BF16)
    moves, ws = fk.alloc_moves(2), fk.alloc_pages_workspace(None)
    moves.copy_(torch.tensor([2, 0, 0, nb - 2, nb - 1, 7], dtype=torch.int32))
    fk.pages_copy(desc, fk.PagePools([k], [v], fk.FUSE_BF16, bs), moves, ws)
    fk.check_errors(ws)
    for i, x in enumerate((k, v)):
        assert (x[nb - 2] == 1 + i).all() and (x[7] == 3 + i).all() and (x[nb - 1] == 3 + i).all()


def test_copy_reports_bad_lists():
    k, v = (torch.randn(8, 16, 2, 64, device="cuda") for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    desc = fk.layer_desc(64, 2, 2, 64, 1e4, fk.FUSE_F32)
    pools, ws = fk.PagePools([k], [v], fk.FUSE_F32, 16), fk.alloc_pages_workspace(None)
    for head in (3, -1):                                     # a count past the list, or negative
        moves = torch.tensor([head, 0, 0, 1, 2, 3], dtype=torch.int32, device="cuda")
        fk.pages_copy(desc, pools, moves, ws)
        with pytest.raises(fk.FuseError) as e:
            fk.check_errors(ws)
        assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
        assert torch.equal(k, k0) and torch.equal(v, v0)
    moves = torch.tensor([3, 0, 0, 8, -1, 1, 2, 3], dtype=torch.int32, device="cuda")
    fk.pages_copy(desc, pools, moves, ws)                    # only the last pair is inside
    with pytest.raises(fk.FuseError):
        fk.check_errors(ws)
    k0[3], v0[3] = k0[2], v0[2]
    assert torch.equal(k, k0) and torch.equal(v, v0)


def _small():
    tab = dev([[0, 5], [3]])
    refs = torch.zeros(8, dtype=torch.int32, device="cuda")
    refs[torch.tensor([0, 5, 3])] = 1
    return tab, [20, 16], refs


def test_fork_refuses_as_a_whole():
    for what in ("outside", "negative", "dead", "full"):
        tab, lens, refs = _small()
        if what == "outside":
            tab[0][1] = 8
        elif what == "negative":
            tab[1][0] = -1
        elif what == "dead":
            refs[3] = 0
        else:
            refs.clamp_(min=1)
        r0 = refs.clone()
        out = dev([[-9, -9], [-9]])
        src, dst = page_table(tab, lens, 16, 8), page_table(out, lens, 16, 8)
        moves, ws = fk.alloc_moves(2), fk.alloc_pages_workspace(src)
        moves.fill_(99)
        fk.pages_fork(src, dst, refs, moves, ws)
        with pytest.raises(fk.FuseError) as e:
            fk.check_errors(ws)
        assert e.value.status == (fk.FUSE_ERR_NO_PAGES if what == "full" else fk.FUSE_ERR_DEVICE_BOUNDS)
        assert torch.equal(refs, r0) and lists(out) == [[-9, -9], [-9]] and int(moves[0]) == 0


def test_compact_refuses_as_a_whole():
    for bad in (8, -1, 6):                                   # outside, negative, a free page
        tab, lens, refs = _small()
        tab[1][0] = bad
        r0, t0 = refs.clone(), lists(tab)
        seqs = page_table(tab, lens, 16, 8)
        moves, ws = fk.alloc_moves(4), fk.alloc_pages_workspace(seqs)
        moves.fill_(99)
        fk.pages_compact(seqs, refs, moves, ws)
        with pytest.raises(fk.FuseError) as e:
            fk.check_errors(ws)
        assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
        assert torch.equal(refs, r0) and lists(tab) == t0 and int(moves[0]) == 0


def test_free_reports_what_was_free_already():
    tab, lens, refs = _small()
    tables = page_table(tab + [tab[1]], lens + [16], 16, 8)      # page 3 given up twice, held once
    ws = fk.alloc_pages_workspace(None)
    fk.pages_free(tables, refs, ws)
    with pytest.raises(fk.FuseError) as e:
        fk.check_errors(ws)
    assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
    assert refs.cpu().tolist() == [0] * 8
    tab[0][0], tab[0][1] = 9, -2
    refs.fill_(2)
    fk.pages_free(page_table(tab, lens, 16, 8), refs, ws)
    with pytest.raises(fk.FuseError):
        fk.check_errors(ws)
    assert refs.cpu().tolist() == [2, 2, 2, 1, 2, 2, 2, 2]


def test_graph_of_fork_copy_and_drop():
    k, v = (torch.randn(64, 16, 2, 64, device="cuda") for _ in range(2))
    desc = fk.layer_desc(64, 2, 2, 64, 1e4, fk.FUSE_F32)
    pools = fk.PagePools([k], [v], fk.FUSE_F32, 16)
    tables, lens, refs = draw(9, 64, 4, 150, 16, share=False)
    d_tab, d_refs = dev(tables), torch.from_numpy(refs).cuda()
    out = [torch.zeros(max(1, -(-n // 16)), dtype=torch.int32, device="cuda") for n in lens]
    src, dst = page_table(d_tab, lens, 16, 64), page_table(out, lens, 16, 64)
    moves, ws = fk.alloc_moves(len(lens)), fk.alloc_pages_workspace(src)

    def go():
        fk.pages_fork(src, dst, d_refs, moves, ws)
        fk.pages_copy(desc, pools, moves, ws)
        fk.pages_free(dst, d_refs, ws)
    go()
    fk.check_errors(ws)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        go()
    for page in range(64):
        k[page].normal_()
    for t in out:
        t.fill_(-9)
    g.replay()
    fk.check_errors(ws)
    want = fork_reference(tables, lens, refs, 16)
    assert [t[:-(-n // 16)] for t, n in zip(lists(out), lens)] == want[0]
    for a, b in want[2]:
        assert torch.equal(k[a], k[b])
    assert d_refs.cpu().tolist() == refs.tolist()


@pytest.mark.parametrize("storage", ["u4", "bf16"])
def test_fork_compact_and_attend_together(storage):
    """A paged batch is forked, its first branch dropped, the pool packed: the
    branches attend as the sequences did, bit for bit."""
    bs = 16
    a = Attend(AttendCase(lens=[[33, 64, 7], [100, 1]], n_query=[4, 6], k=[20, 11], storage=storage,
                          paged=True, block_size=bs, heads=(8, 2, 128), spare_blocks=9))
    want = a.run().clone()
    fk.check_errors(a.ws)
    flat = [n for x in a.c.lens for n in x]
    nb = a.n_blocks
    grow = lambda x: None if x is None else torch.cat([x, torch.zeros_like(x)])  # noqa: E731
    a.K, a.V, a.vs, a.vz = (grow(x) for x in (a.K, a.V, a.vs, a.vz))
    a.n_blocks = 2 * nb
    refs = torch.zeros(2 * nb, dtype=torch.int32, device="cuda")
    for t in a.tables:
        refs[t.long()] += 1
    src = page_table(a.tables, flat, bs, 2 * nb)
    out = [torch.zeros_like(t) for t in a.tables]
    dst = page_table(out, flat, bs, 2 * nb)
    moves, ws = fk.alloc_moves(nb), fk.alloc_pages_workspace(src)
    pools = fk.PagePools([a.K], [a.V], cache_ops.KIND[storage], bs, [a.vs] if storage == "u4" else [],
                         [a.vz] if storage == "u4" else [])
    fk.pages_fork(src, dst, refs, moves, ws)
    fk.pages_copy(a.desc, pools, moves, ws)
    fk.pages_free(src, refs, ws)
    fk.pages_compact(dst, refs, moves, ws)
    fk.pages_copy(a.desc, pools, moves, ws)
    fk.check_errors(ws)
    n = sum(-(-x // bs) for x in flat)
    assert int(moves[1]) == n and (refs[:n] == 1).all() and (refs[n:] == 0).all()
    a.chunks = a.table(out)
    a.O.zero_()
    assert torch.equal(a.run(), want)
    fk.check_errors(a.ws)


def test_prompt_quantize_attend_together():
    """The whole run: chunks attend to themselves, their caches become 4-bit
    codes, and a new token attends over the codes and its own row."""
    Hq, Hkv, d, base = 8, 2, 128, 1e4
    lens, g = [48, 80], torch.Generator().manual_seed(5)
    T = sum(lens)
    desc = fk.layer_desc(64, Hq, Hkv, d, base, fk.FUSE_BF16)
    mk = lambda n, h: torch.randn(n, h, d, generator=g).bfloat16().cuda()  # noqa: E731
    Q, K, V = mk(T, Hq), mk(T, Hkv), mk(T, Hkv)
    O = torch.zeros_like(Q)
    each = fk.plan_requests(lens, [0] * len(lens), 0.0)
    ws = fk.alloc_workspace(desc, each)
    fk.attend_prompt(desc, each, Q, K, V, O, ws)
    fk.check_errors(ws)
    O_ref, O_tol = cache_ops.prompt_reference(Q, K, V, [(0, 48), (48, 80)], "bf16")
    assert (np.abs(f64(O) - O_ref) <= O_tol).all()
    codes = {n: torch.zeros(T, Hkv, d // 2, dtype=torch.uint8, device="cuda") for n in "kv"}
    ks, kz = (torch.zeros(2, Hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    vs, vz = (torch.zeros(T, Hkv, dtype=torch.float16, device="cuda") for _ in range(2))
    a, b, at = [], [], 0
    for i, n in enumerate(lens):
        e, q = fk.Chunk(), fk.Chunk()
        e.k, e.v = K[at:].data_ptr(), V[at:].data_ptr()
        q.k, q.v = codes["k"][at:].data_ptr(), codes["v"][at:].data_ptr()
        q.k_scale, q.k_zero = ks[i].data_ptr(), kz[i].data_ptr()
        q.v_scale, q.v_zero = vs[at:].data_ptr(), vz[at:].data_ptr()
        for x in (e, q):
            x.dst_row, x.pos, x.len = at, at, n
        a.append(e)
        b.append(q)
        at += n
    src = fk.ChunkTable(a, fk.FUSE_KV_CONTIGUOUS, fk.FUSE_BF16)
    dst = fk.ChunkTable(b, fk.FUSE_KV_CONTIGUOUS, fk.FUSE_U4_ASYM)
    fk.kivi_quantize(desc, src, dst)
    reqs = fk.plan_requests([T], [1], 0.0)
    q1, k1, v1 = mk(1, Hq), mk(1, Hkv), mk(1, Hkv)
    o1 = torch.zeros_like(q1)
    ws2 = fk.alloc_attend_workspace(desc, dst, reqs, 1)
    fk.attend_chunks(desc, dst, reqs, 1, q1, None, k1, v1, o1, ws2)
    fk.check_errors(ws2)
    # the same through the stitched fp32 cache
    d32 = fk.layer_desc(64, Hq, Hkv, d, base, fk.FUSE_F32)
    Kf, Vf = (torch.zeros(T + 1, Hkv, d, device="cuda") for _ in range(2))
    ws3 = fk.alloc_workspace(d32, reqs)
    fk.stitch_rerotate(d32, dst, Kf, Vf, ws3)
    fk.check_errors(ws3)
    Kf[T], Vf[T] = k1[0].float(), v1[0].float()
    for h in range(Hq):
        k, v = f64(Kf[:, h // 4]), f64(Vf[:, h // 4])
        o, A, S = cache_ops.attention(f64(q1[0, h]), k, v)
        # codes of 4 bits: zero and scaled part are at most 3 times a key's span each
        e = 8 * S * ((d + 16) * 2.0 ** -23 + 2.0 ** -20)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -9 + 2 * e) * A
        assert (np.abs(f64(o1[0, h]) - o) <= tol).all()


@pytest.mark.parametrize("call", ["fork", "compact"])
@pytest.mark.parametrize("n_blocks,page", [(8, 1), (8, 7), (9, 8), (33003, 4), (33003, 33002), (33003, 20000)])
def test_a_negative_count_is_refused_as_a_whole(call, n_blocks, page):
    """A page whose count is negative and that no table names: below the live
    pages' number it would leave fewer holes than pages to move."""
    top = n_blocks - 2 if page == n_blocks - 1 else n_blocks - 1
    tab, lens = dev([[0, top], [3]]), [20, 16]
    refs = torch.zeros(n_blocks, dtype=torch.int32, device="cuda")
    refs[torch.tensor([0, top, 3])] = 1
    refs[page] = -1
    r0, t0 = refs.clone(), lists(tab)
    out = dev([[-9, -9], [-9]])
    src, dst = page_table(tab, lens, 16, n_blocks), page_table(out, lens, 16, n_blocks)
    moves, ws = fk.alloc_moves(n_blocks // 2), fk.alloc_pages_workspace(src)
    moves.fill_(99)
    if call == "fork":
        fk.pages_fork(src, dst, refs, moves, ws)
    else:
        fk.pages_compact(src, refs, moves, ws)
    with pytest.raises(fk.FuseError) as e:
        fk.check_errors(ws)
    assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
    assert torch.equal(refs, r0) and lists(tab) == t0 and lists(out) == [[-9, -9], [-9]]
    assert int(moves[0]) == 0 and (moves[2:] == 99).all()
