"""Refusals of the cache operators, found on the host before any launch: no
GPU is needed, and no call here reaches one."""

import ctypes

import pytest
import torch

A = 1 << 20                                # an aligned stand-in, never dereferenced


@pytest.fixture(scope="module")
def fk():
    from rag_kv_cache_rerotate_gb300 import _build, fusekv
    _build.build()
    fusekv.load()
    return fusekv


def _desc(fk, **kw):
    a = dict(hidden=64, n_q_heads=8, n_kv_heads=2, head_dim=128, rope_base=1e4, dtype=fk.FUSE_BF16)
    a.update(kw)
    return fk.layer_desc(**a)


def _chunks(fk, spans, storage=None, **kw):
    es = []
    for row, n in spans:
        e = fk.Chunk()
        e.k = e.v = e.k_scale = e.k_zero = e.v_scale = e.v_zero = A
        e.block_table = A
        e.dst_row, e.len = row, n
        es.append(e)
    t = fk.ChunkTable(es, kw.get("layout", fk.FUSE_KV_CONTIGUOUS),
                      fk.FUSE_U4_ASYM if storage is None else storage, kw.get("bs", 0),
                      kw.get("nb", 0), device=None)
    t.c.d_chunks = A
    return t


def _reqs(fk, reqs):
    t = fk.RequestTable([fk.Request(*r) for r in reqs], device=None)
    t.c.d_req = A
    return t


def _attend(fk, desc, chunks, reqs, n_new=1, Q=A, idx=A, Ks=A, Vs=A, O=A, ws=A, nbytes=1 << 40):
    return fk.load().fuse_attend_chunks(ctypes.byref(desc), ctypes.byref(chunks.c) if chunks else None,
                                        ctypes.byref(reqs.c) if reqs else None, n_new, Q, idx, Ks, Vs,
                                        O, ws, nbytes, None)


ONE = [(0, 0, 0, 0, 100, 5, 3, 0)]


def test_attend_refuses_missing_and_misaligned_pointers(fk):
    d, c, r = _desc(fk), _chunks(fk, [(0, 60), (60, 40)]), _reqs(fk, ONE)
    need = fk.attend_workspace_size(d, c, r, 1)
    for name in ("Q", "Ks", "Vs", "O", "idx"):
        assert _attend(fk, d, c, r, **{name: None}) == fk.FUSE_ERR_INVALID_ARG, name
        assert _attend(fk, d, c, r, **{name: A + (2 if name == "idx" else 8)}) == fk.FUSE_ERR_MISALIGNED, name
    assert _attend(fk, d, None, r) == fk.FUSE_ERR_INVALID_ARG
    assert _attend(fk, d, c, None) == fk.FUSE_ERR_INVALID_ARG
    assert _attend(fk, d, c, r, ws=None) == fk.FUSE_ERR_WORKSPACE
    assert _attend(fk, d, c, r, nbytes=need - 1) == fk.FUSE_ERR_WORKSPACE
    assert _attend(fk, d, c, r, ws=A + 16) == fk.FUSE_ERR_MISALIGNED
    empty = _reqs(fk, [])
    assert _attend(fk, d, _chunks(fk, []), empty) == fk.FUSE_OK           # nothing to do


def test_attend_refuses_what_it_does_not_take(fk):
    c, r = _chunks(fk, [(0, 100)]), _reqs(fk, ONE)
    for n_new in (0, -1, 9):
        assert _attend(fk, _desc(fk), c, r, n_new) == fk.FUSE_ERR_INVALID_ARG
    assert _attend(fk, _desc(fk), c, r, 6) == fk.FUSE_ERR_INVALID_ARG     # more than the query tokens
    assert _attend(fk, _desc(fk, head_dim=96), c, r) == fk.FUSE_ERR_UNSUPPORTED
    assert _attend(fk, _desc(fk, n_q_heads=6), c, r) == fk.FUSE_ERR_UNSUPPORTED      # 3 heads a KV head
    other = _chunks(fk, [(0, 100)], fk.FUSE_F32)                          # not the layer's type
    assert _attend(fk, _desc(fk), other, r) == fk.FUSE_ERR_UNSUPPORTED
    none = _chunks(fk, [(0, 100)])
    none.host[0].v_zero = None
    assert _attend(fk, _desc(fk), none, r) == fk.FUSE_ERR_INVALID_ARG
    paged = _chunks(fk, [(0, 100)], layout=fk.FUSE_KV_PAGED, bs=16, nb=8)
    paged.host[0].block_table = None
    assert _attend(fk, _desc(fk), paged, r) == fk.FUSE_ERR_INVALID_ARG


@pytest.mark.parametrize("spans", [[(40, 60), (0, 40)], [(0, 50), (49, 20)], [(90, 20)], [(101, 4)],
                                   [(0, 100), (105, 8)], [(1000, 5)]])
def test_attend_refuses_chunks_outside_a_context(fk, spans):
    r = _reqs(fk, ONE)
    assert _attend(fk, _desc(fk), _chunks(fk, spans), r) == fk.FUSE_ERR_INVALID_ARG
    with pytest.raises(fk.FuseError):
        fk.attend_workspace_size(_desc(fk), _chunks(fk, spans), r, 1)


def test_attend_refuses_requests_out_of_row_order(fk):
    r = _reqs(fk, [(105, 0, 0, 0, 10, 5, 0, 0), (0, 0, 0, 5, 100, 5, 0, 0)])
    assert _attend(fk, _desc(fk), _chunks(fk, [(0, 10)]), r) == fk.FUSE_ERR_INVALID_ARG


def test_attend_workspace_grows_with_the_new_tokens(fk):
    d, c, r = _desc(fk), _chunks(fk, [(0, 100)]), _reqs(fk, ONE)
    assert fk.attend_workspace_size(d, c, r, 5) >= fk.attend_workspace_size(d, c, r, 1) > 256


def test_prompt_refusals(fk):
    d = _desc(fk)
    r = _reqs(fk, [(0, 0, 0, 0, 100, 5, 0, 0), (105, 0, 0, 0, 3, 0, 0, 0)])

    def call(reqs=r, Q=A, K=A, V=A, O=A, ws=A, n=1 << 20, desc=d):
        return fk.load().fuse_attend_prompt(ctypes.byref(desc), ctypes.byref(reqs.c) if reqs else None,
                                            Q, K, V, O, ws, n, None)
    for name in "QKVO":
        assert call(**{name: None}) == fk.FUSE_ERR_INVALID_ARG
        assert call(**{name: A + 8}) == fk.FUSE_ERR_MISALIGNED
    assert call(reqs=None) == fk.FUSE_ERR_INVALID_ARG
    assert call(ws=None) == fk.FUSE_ERR_WORKSPACE
    assert call(n=255) == fk.FUSE_ERR_WORKSPACE
    assert call(ws=A + 64) == fk.FUSE_ERR_MISALIGNED
    assert call(desc=_desc(fk, head_dim=32)) == fk.FUSE_ERR_UNSUPPORTED
    late = _reqs(fk, [(50, 0, 0, 0, 10, 0, 0, 0), (0, 0, 0, 0, 10, 0, 0, 0)])
    assert call(reqs=late) == fk.FUSE_ERR_INVALID_ARG                     # row order
    over = _reqs(fk, [(0, 0, 0, 0, 10, 0, 0, 0), (9, 0, 0, 0, 10, 0, 0, 0)])
    assert call(reqs=over) == fk.FUSE_ERR_INVALID_ARG                     # shared rows
    assert call(reqs=_reqs(fk, [(0, 0, 0, 0, 0, 0, 0, 0)])) == fk.FUSE_OK  # no row at all


def _tables(fk, lens, bs=16, nb=8, **kw):
    return _chunks(fk, [(0, n) for n in lens], fk.FUSE_BF16, layout=kw.get("layout", fk.FUSE_KV_PAGED),
                   bs=bs, nb=nb)


def test_fork_refusals(fk):
    def call(src, dst, refs=A, moves=A, cap=4, ws=A, n=1 << 30):
        return fk.load().fuse_pages_fork(ctypes.byref(src.c), ctypes.byref(dst.c), refs, moves, cap, ws,
                                         n, None)

    def other(lens, **kw):                              # destination tables elsewhere
        t = _tables(fk, lens, **kw)
        for i in range(len(lens)):
            t.host[i].block_table = 2 * A
        return t
    s = _tables(fk, [20, 16])
    assert call(s, _tables(fk, [20, 16])) == fk.FUSE_ERR_INVALID_ARG     # dst is the source table
    assert call(s, other([20])) == fk.FUSE_ERR_INVALID_ARG
    assert call(s, other([20, 17])) == fk.FUSE_ERR_INVALID_ARG
    assert call(s, other([20, 16], bs=8)) == fk.FUSE_ERR_INVALID_ARG
    assert call(s, other([20, 16], nb=9)) == fk.FUSE_ERR_INVALID_ARG
    assert call(_tables(fk, [20], layout=fk.FUSE_KV_CONTIGUOUS), other([20])) == fk.FUSE_ERR_UNSUPPORTED
    d = other([20, 16])
    assert call(s, d, refs=None) == fk.FUSE_ERR_INVALID_ARG
    assert call(s, d, moves=None) == fk.FUSE_ERR_INVALID_ARG
    assert call(s, d, cap=-1) == fk.FUSE_ERR_INVALID_ARG
    assert call(s, d, cap=0) == fk.FUSE_ERR_WORKSPACE                     # one partly filled page
    assert call(s, d, refs=A + 4) == fk.FUSE_ERR_MISALIGNED
    assert call(s, d, moves=A + 2) == fk.FUSE_ERR_MISALIGNED
    assert call(s, d, n=256) == fk.FUSE_ERR_WORKSPACE
    d.host[1].block_table = None
    assert call(s, d) == fk.FUSE_ERR_INVALID_ARG
    d.host[1].block_table = A + 2
    assert call(s, d) == fk.FUSE_ERR_MISALIGNED


def test_free_and_compact_refusals(fk):
    lib, t = fk.load(), _tables(fk, [20, 16])

    def free(t=t, refs=A, ws=A, n=256):
        return lib.fuse_pages_free(ctypes.byref(t.c), refs, ws, n, None)

    def compact(t=t, refs=A, moves=A, cap=4, ws=A, n=1 << 30):
        return lib.fuse_pages_compact(ctypes.byref(t.c), refs, moves, cap, ws, n, None)
    assert free(refs=None) == fk.FUSE_ERR_INVALID_ARG
    assert free(refs=A + 8) == fk.FUSE_ERR_MISALIGNED
    assert free(n=255) == fk.FUSE_ERR_WORKSPACE
    assert free(_tables(fk, [])) == fk.FUSE_OK                            # nothing to drop
    assert compact(refs=None) == fk.FUSE_ERR_INVALID_ARG
    assert compact(moves=None) == fk.FUSE_ERR_INVALID_ARG
    assert compact(cap=3) == fk.FUSE_ERR_WORKSPACE                        # 8 pages may need 4 moves
    assert compact(n=300) == fk.FUSE_ERR_WORKSPACE
    assert compact(_tables(fk, [20], nb=0)) == fk.FUSE_ERR_INVALID_ARG
    assert compact(_tables(fk, [20], bs=0)) == fk.FUSE_ERR_INVALID_ARG
    assert compact(_tables(fk, [-1])) == fk.FUSE_ERR_INVALID_ARG
    assert compact(_tables(fk, [20], nb=1 << 30)) == fk.FUSE_ERR_UNSUPPORTED


def test_copy_refusals(fk):
    lib = fk.load()

    def call(desc=None, kind=None, bs=16, nb=8, n_pools=1, reserved=0, k=A, v=A, s=A, z=A, moves=A,
             cap=4, ws=A, n=256):
        pool = (fk.Pool * 1)(fk.Pool(k, v, s, z))
        p = fk.Pools(n_pools, fk.FUSE_U4_ASYM if kind is None else kind, bs, reserved, nb,
                     ctypes.addressof(pool))
        return lib.fuse_pages_copy(ctypes.byref(desc or _desc(fk)), ctypes.byref(p), moves, cap, ws, n, None)
    assert call(k=None) == fk.FUSE_ERR_INVALID_ARG
    assert call(z=None) == fk.FUSE_ERR_INVALID_ARG
    assert call(v=A + 8) == fk.FUSE_ERR_MISALIGNED
    assert call(s=A + 1) == fk.FUSE_ERR_MISALIGNED
    assert call(moves=None) == fk.FUSE_ERR_INVALID_ARG
    assert call(moves=A + 1) == fk.FUSE_ERR_MISALIGNED
    assert call(cap=-1) == fk.FUSE_ERR_INVALID_ARG
    assert call(kind=7) == fk.FUSE_ERR_INVALID_ARG
    assert call(bs=0) == fk.FUSE_ERR_INVALID_ARG
    assert call(nb=0) == fk.FUSE_ERR_INVALID_ARG
    assert call(nb=1 << 40) == fk.FUSE_ERR_UNSUPPORTED
    assert call(reserved=1) == fk.FUSE_ERR_INVALID_ARG
    assert call(n=255) == fk.FUSE_ERR_WORKSPACE
    assert call(bs=1 << 30) == fk.FUSE_ERR_UNSUPPORTED
    assert call(cap=0) == fk.FUSE_OK and call(n_pools=0) == fk.FUSE_OK    # nothing to copy


def test_binding_refuses_wrong_tensors(fk):
    d, c, r = _desc(fk), _chunks(fk, [(0, 100)]), _reqs(fk, ONE)
    bf, ws = torch.bfloat16, torch.zeros(256, dtype=torch.uint8)
    Q, S = torch.zeros(1, 8, 128, dtype=bf), torch.zeros(8, 2, 128, dtype=bf)
    idx = torch.zeros(3, dtype=torch.int32)

    def call(Q=Q, idx=idx, Ks=S, Vs=S, O=Q):
        with pytest.raises(ValueError):
            fk.attend_chunks(d, c, r, 1, Q, idx, Ks, Vs, O, ws)
    call(Q=Q.float())
    call(Q=torch.zeros(2, 8, 128, dtype=bf))
    call(O=torch.zeros(1, 8, 256, dtype=bf)[:, :, ::2])
    call(idx=idx.long())
    call(idx=idx[:2])
    call(idx=None)
    call(Ks=S[:7])
    call(Vs=torch.zeros(8, 2, 64, dtype=bf))
    grown = _reqs(fk, ONE)
    grown.extents()
    grown.host[0].n_query += 4                             # the table is looked at again
    with pytest.raises(ValueError):
        fk.attend_chunks(d, c, grown, 1, Q, idx, S, S, Q, ws)
    with pytest.raises(ValueError):
        fk.attend_chunks(d, c, r, 1, Q, idx, S, S, Q, ws[::2])
    with pytest.raises(ValueError):
        fk.attend_prompt(d, r, torch.zeros(104, 8, 128, dtype=bf), torch.zeros(105, 2, 128, dtype=bf),
                         torch.zeros(105, 2, 128, dtype=bf), torch.zeros(105, 8, 128, dtype=bf), ws)
    with pytest.raises(ValueError):
        fk.pages_compact(_tables(fk, [20]), torch.zeros(7, dtype=torch.int32), torch.zeros(10, dtype=torch.int32), ws)
    with pytest.raises(ValueError):
        fk.pages_free(_tables(fk, [20]), torch.zeros(8), ws)
    with pytest.raises(ValueError):
        fk.PagePools([torch.zeros(8, 16, 2, 128)], [torch.zeros(8, 16, 2, 64)], fk.FUSE_F32, 16)


def test_request_table_device_copy_follows_the_host_table(fk):
    t = fk.RequestTable([fk.Request(*r) for r in ONE], device="cpu")
    assert bytes(t.dev.numpy()) == bytes(t.host)
    t.host[0].n_query += 4
    t.update()
    assert bytes(t.dev.numpy()) == bytes(t.host) and t.extents().n_tok == 109
    t.host[0].n_query -= 1
    S = torch.zeros(12, 2, 128, dtype=torch.bfloat16)
    Q = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(fk.FuseError):                      # refused: no workspace to speak of
        fk.attend_chunks(_desc(fk), _chunks(fk, [(0, 100)]), t, 1, Q, torch.zeros(3, dtype=torch.int32), S, S, Q,
                         torch.zeros(0, dtype=torch.uint8))
    assert bytes(t.dev.numpy()) == bytes(t.host)           # the call brought the copy up to date first


@pytest.mark.parametrize("heads,n_new", [((32, 8), 1), ((64, 8), 8), ((4, 2), 1), ((3, 3), 1)])
@pytest.mark.parametrize("long,short,n", [(8192, 32, 500), (32768, 16, 2000), (4096, 1, 4000)])
def test_attend_workspace_does_not_grow_with_the_longest_chunk(fk, heads, n_new, long, short, n):
    # one long chunk beside short ones takes what as many equal ones of the same
    # tokens take, but for the short ones' partly filled segments
    d = _desc(fk, n_q_heads=heads[0], n_kv_heads=heads[1])
    total = long + short * n

    def size(lens):
        spans, at = [], 0
        for x in lens:
            spans.append((at, x))
            at += x
        r = _reqs(fk, [(0, 0, 0, 0, at, n_new, 0, 0)])
        return fk.attend_workspace_size(d, _chunks(fk, spans), r, n_new)
    assert size([short] * (n // 2) + [long] + [short] * (n - n // 2)) <= 1.5 * size([total // n] * n)


@pytest.mark.parametrize("n,long", [(1000, 30000), (200, 4096)])
def test_attend_workspace_does_not_grow_with_the_longest_generation(fk, n, long):
    # requests that have generated little beside one that has generated much
    d = _desc(fk, n_q_heads=32, n_kv_heads=8)

    def size(queries):
        reqs, row, out = [], 0, 0
        for q in queries:
            reqs.append((row, 0, 0, out, 0, q, 0, 0))
            row, out = row + q, out + q
        return fk.attend_workspace_size(d, _chunks(fk, []), _reqs(fk, reqs), 1)
    assert size([2] * (n // 2) + [long] + [2] * (n // 2)) <= 1.5 * size([2 + long // n] * n)
