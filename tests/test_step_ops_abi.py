"""Refusals of the operators of a speculative step, found on the host before
any launch: no GPU is needed, and no call here reaches one."""

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


def _seqs(fk, **kw):
    a = dict(n_seq=3, block_size=16, max_blocks=8, max_new=4, n_pool_blocks=30, tables=A, lens=A, rows=A)
    a.update(kw)
    return fk.Seqs(**a)


BAD_SEQS = [("n_seq", -1, "INVALID_ARG"), ("n_seq", 65536, "UNSUPPORTED"), ("block_size", 0, "INVALID_ARG"),
            ("max_blocks", 0, "INVALID_ARG"), ("max_new", 0, "INVALID_ARG"), ("max_new", 65, "UNSUPPORTED"),
            ("n_pool_blocks", 0, "INVALID_ARG"), ("max_blocks", 1 << 28, "UNSUPPORTED"),
            ("max_blocks", (1 << 27) - 15, "UNSUPPORTED"), ("n_pool_blocks", (1 << 27) - 15, "UNSUPPORTED"),
            ("tables", None, "INVALID_ARG"), ("lens", None, "INVALID_ARG"), ("rows", None, "INVALID_ARG"),
            ("tables", A + 2, "MISALIGNED"), ("lens", A + 1, "MISALIGNED"), ("rows", A + 2, "MISALIGNED")]


def _append(fk, desc=None, rope=None, seqs=None, n_rows=9, parents=A, ws=A, nbytes=256, **io):
    x = dict(Q=A, K=A, V=A, q_stride=1024, k_stride=256, v_stride=256, Qr=A, Kr=A, k_pool=A, v_pool=A)
    x.update(io)
    r = lambda v: ctypes.byref(v) if v is not None else None  # noqa: E731
    return fk.load().fuse_cache_append(r(desc or _desc(fk)), r(rope if rope is not None else fk.rope_desc()),
                                       r(seqs or _seqs(fk)), n_rows, parents, r(fk.Append(**x)), ws, nbytes, None)


def test_append_refusals(fk):
    for name in ("K", "V", "k_pool", "v_pool", "Q", "Qr"):             # Q and Qr go together
        assert _append(fk, **{name: None}) == fk.FUSE_ERR_INVALID_ARG, name
    for name in ("Q", "K", "V", "Qr", "Kr", "k_pool", "v_pool"):
        assert _append(fk, **{name: A + 8}) == fk.FUSE_ERR_MISALIGNED, name
    assert _append(fk, parents=A + 2) == fk.FUSE_ERR_MISALIGNED
    assert _append(fk, k_stride=255) == fk.FUSE_ERR_INVALID_ARG        # rows overlap
    assert _append(fk, q_stride=1028) == fk.FUSE_ERR_MISALIGNED        # 8 bytes past 16
    assert _append(fk, v_stride=260) == fk.FUSE_ERR_MISALIGNED
    assert _append(fk, ws=None) == fk.FUSE_ERR_WORKSPACE
    assert _append(fk, nbytes=255) == fk.FUSE_ERR_WORKSPACE
    assert _append(fk, ws=A + 16) == fk.FUSE_ERR_MISALIGNED
    assert _append(fk, n_rows=-1) == fk.FUSE_ERR_INVALID_ARG
    assert _append(fk, n_rows=1 << 31) == fk.FUSE_ERR_UNSUPPORTED
    assert _append(fk, desc=_desc(fk, head_dim=96)) == fk.FUSE_ERR_UNSUPPORTED
    # nothing to do
    assert _append(fk, n_rows=0) == fk.FUSE_OK
    assert _append(fk, seqs=_seqs(fk, n_seq=0)) == fk.FUSE_OK
    for name, value, status in BAD_SEQS:
        assert _append(fk, seqs=_seqs(fk, **{name: value})) == getattr(fk, "FUSE_ERR_" + status), name


def test_rope_refusals(fk):
    bad = [(dict(layout=2), "INVALID_ARG"), (dict(rot_dim=-16), "INVALID_ARG"), (dict(rot_dim=144), "INVALID_ARG"),
           (dict(rot_dim=24), "UNSUPPORTED"), (dict(scaling=4), "INVALID_ARG"), (dict(mscale=0.0), "INVALID_ARG"),
           (dict(mscale=float("nan")), "INVALID_ARG"),
           (dict(scaling=fk.FUSE_ROPE_LINEAR, factor=0.5), "INVALID_ARG"),
           (dict(scaling=fk.FUSE_ROPE_LLAMA3, factor=8.0, low=1.0, high=4.0), "INVALID_ARG"),      # no length
           (dict(scaling=fk.FUSE_ROPE_YARN, factor=4.0, original_len=4096, low=2.0, high=1.0), "INVALID_ARG"),
           (dict(scaling=fk.FUSE_ROPE_YARN, factor=4.0, original_len=4096, low=0.0, high=1.0), "INVALID_ARG")]
    for kw, status in bad:
        assert _append(fk, rope=fk.rope_desc(**kw)) == getattr(fk, "FUSE_ERR_" + status), kw


def test_tree_refusals(fk):
    def call(desc=None, seqs=None, n_rows=9, parents=A, Q=A, k=A, v=A, O=A, ws=A, n=1 << 40):
        return fk.load().fuse_attend_tree(ctypes.byref(desc or _desc(fk)), ctypes.byref(seqs or _seqs(fk)), n_rows,
                                          parents, Q, k, v, O, ws, n, None)
    for name in "QkvO":
        assert call(**{name: None}) == fk.FUSE_ERR_INVALID_ARG
        assert call(**{name: A + 8}) == fk.FUSE_ERR_MISALIGNED
    assert call(parents=A + 2) == fk.FUSE_ERR_MISALIGNED
    assert call(ws=None) == fk.FUSE_ERR_WORKSPACE
    assert call(ws=A + 64) == fk.FUSE_ERR_MISALIGNED
    need = ctypes.c_size_t(0)
    size = fk.load().fuse_tree_workspace_size
    assert size(ctypes.byref(_desc(fk)), ctypes.byref(_seqs(fk)), ctypes.byref(need)) == fk.FUSE_OK
    assert call(n=need.value - 1) == fk.FUSE_ERR_WORKSPACE
    assert call(n_rows=0) == fk.FUSE_OK
    assert call(seqs=_seqs(fk, n_seq=0)) == fk.FUSE_OK
    for name, value, status in BAD_SEQS:
        assert call(seqs=_seqs(fk, **{name: value})) == getattr(fk, "FUSE_ERR_" + status), name
    assert call(desc=_desc(fk, n_q_heads=6)) == fk.FUSE_ERR_UNSUPPORTED
    assert size(ctypes.byref(_desc(fk)), None, ctypes.byref(need)) == fk.FUSE_ERR_INVALID_ARG
    assert size(ctypes.byref(_desc(fk)), ctypes.byref(_seqs(fk)), None) == fk.FUSE_ERR_INVALID_ARG


def test_verify_refusals(fk):
    def call(n_seq=2, n_rows=9, vocab=100, rows=A, parents=A, tokens=A, P=A, p_stride=100, Q=A, q_stride=100, u=A,
             u_next=A, max_path=8, path=A, count=A, next=A, ws=A, n=256):
        return fk.load().fuse_verify_tree(n_seq, n_rows, vocab, rows, parents, tokens, P, p_stride, Q, q_stride, u,
                                          u_next, max_path, path, count, next, ws, n, None)
    for name in ("rows", "parents", "tokens", "P", "u", "u_next", "path", "count", "next"):
        assert call(**{name: None}) == fk.FUSE_ERR_INVALID_ARG, name
        assert call(**{name: A + 2}) == fk.FUSE_ERR_MISALIGNED, name
    assert call(Q=A + 2) == fk.FUSE_ERR_MISALIGNED
    for kw in (dict(n_seq=-1), dict(n_rows=-1), dict(vocab=0), dict(max_path=0), dict(p_stride=99), dict(q_stride=99)):
        assert call(**kw) == fk.FUSE_ERR_INVALID_ARG, kw
    for kw in (dict(n_seq=65536), dict(max_path=65), dict(vocab=1 << 30, p_stride=1 << 31, q_stride=1 << 31)):
        assert call(**kw) == fk.FUSE_ERR_UNSUPPORTED, kw
    assert call(ws=None) == fk.FUSE_ERR_WORKSPACE
    assert call(n=255) == fk.FUSE_ERR_WORKSPACE
    assert call(n_seq=0) == fk.FUSE_OK


def test_keep_refusals(fk):
    pool = (fk.Pool * 2)(fk.Pool(A, 2 * A, None, None), fk.Pool(3 * A, 4 * A, None, None))

    def pools(**kw):
        a = dict(n_pools=1, kv_storage=fk.FUSE_BF16, block_size=16, reserved=0, n_blocks=30,
                 h_pools=ctypes.addressof(pool))
        a.update(kw)
        return fk.Pools(**a)

    def call(p=None, seqs=None, path=A, max_path=4, count=A, ws=A, n=256):
        return fk.load().fuse_cache_keep(ctypes.byref(_desc(fk)), ctypes.byref(p or pools()),
                                         ctypes.byref(seqs or _seqs(fk)), path, max_path, count, ws, n, None)
    assert call(pools(kv_storage=fk.FUSE_U8_ASYM)) == fk.FUSE_ERR_UNSUPPORTED
    assert call(pools(kv_storage=fk.FUSE_F32)) == fk.FUSE_ERR_UNSUPPORTED          # not the layer's type
    for kw in (dict(block_size=32), dict(n_blocks=31), dict(n_pools=-1), dict(reserved=1), dict(h_pools=None)):
        assert call(pools(**kw)) == fk.FUSE_ERR_INVALID_ARG, kw
    assert call(path=None) == fk.FUSE_ERR_INVALID_ARG
    assert call(count=None) == fk.FUSE_ERR_INVALID_ARG
    assert call(path=A + 2) == fk.FUSE_ERR_MISALIGNED
    assert call(max_path=0) == fk.FUSE_ERR_INVALID_ARG
    assert call(max_path=65) == fk.FUSE_ERR_UNSUPPORTED
    assert call(ws=None) == fk.FUSE_ERR_WORKSPACE
    assert call(seqs=_seqs(fk, n_seq=0)) == fk.FUSE_OK
    for name, value, status in BAD_SEQS:
        assert call(seqs=_seqs(fk, **{name: value})) == getattr(fk, "FUSE_ERR_" + status), name
    assert call(pools(n_pools=2), seqs=_seqs(fk, n_seq=0)) == fk.FUSE_OK
    for name, value in (("k", A), ("k", 2 * A), ("v", A), ("v", 2 * A), ("v", 3 * A)):    # moved twice
        saved = getattr(pool[1], name)
        setattr(pool[1], name, value)
        assert call(pools(n_pools=2)) == fk.FUSE_ERR_INVALID_ARG, (name, value)
        setattr(pool[1], name, saved)
    pool[0].v = None
    assert call() == fk.FUSE_ERR_INVALID_ARG
    pool[0].v = A + 8
    assert call() == fk.FUSE_ERR_MISALIGNED


def test_binding_refuses_what_a_pointer_hides(fk):
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="tables"):
        fk.Sequences(z(3), z(3), z(4), 16, 8, 4)
    with pytest.raises(ValueError, match="lens"):
        fk.Sequences(z(3, 2), z(4), z(4), 16, 8, 4)
    with pytest.raises(ValueError, match="rows"):
        fk.Sequences(z(3, 2), z(3), z(3), 16, 8, 4)
    with pytest.raises(ValueError, match="lens"):
        fk.Sequences(z(3, 2), z(3, dt=torch.int64), z(4), 16, 8, 4)
    if torch.cuda.is_available():
        return                             # the tensors below are host tensors
    seqs = fk.Sequences(z(3, 2), z(3), z(4), 16, 8, 4)
    d, ws = _desc(fk), z(256, dt=torch.uint8)
    b = lambda *s: z(*s, dt=torch.bfloat16)  # noqa: E731
    k, pool = b(5, 2, 128), b(8, 16, 2, 128)

    def append(**kw):
        a = dict(parents=z(5), Q=b(5, 8, 128), K=k, V=k, Qr=b(5, 8, 128), Kr=None, k_pool=pool, v_pool=pool)
        a.update(kw)
        fk.cache_append(d, fk.rope_desc(), seqs, ws=ws, **a)
    for kw, name in ((dict(K=b(5, 2, 64)), "K"), (dict(V=k.float()), "V"), (dict(Qr=None), "Q"),
                     (dict(Qr=b(6, 8, 128)), "Qr"), (dict(parents=z(4)), "parents"), (dict(k_pool=b(8, 8, 2, 128)), "k_pool"),
                     (dict(v_pool=b(7, 16, 2, 128)), "v_pool"), (dict(V=b(5, 128, 2).transpose(1, 2)), "V")):
        with pytest.raises(ValueError, match=name):
            append(**kw)
    with pytest.raises(ValueError, match="O"):
        fk.attend_tree(d, seqs, None, b(5, 8, 128), pool, pool, b(5, 8, 64), ws)
    f = lambda *s: z(*s, dt=torch.float32)  # noqa: E731
    good = dict(rows=z(3), parents=z(5), tokens=z(5), P=f(5, 40), Qd=None, u=f(5), u_next=f(2), path=z(2, 4), count=z(2),
                next=z(2), ws=ws)
    for kw, name in ((dict(P=f(5, 40).double()), "P"), (dict(P=f(40, 5).t()), "P"), (dict(Qd=f(5, 41)), "Qd"),
                     (dict(tokens=z(4)), "tokens"), (dict(u=f(4)), "u"), (dict(path=z(3, 4)), "path"),
                     (dict(next=z(1)), "next")):
        with pytest.raises(ValueError, match=name):
            fk.verify_tree(**{**good, **kw})
    pools = fk.PagePools([pool], [pool], fk.FUSE_BF16, 16)
    with pytest.raises(ValueError, match="count"):
        fk.cache_keep(d, pools, seqs, z(3, 4), z(2), ws)


def test_mscale_is_a_float(fk):
    for x in (1e-60, 1e60, float("inf"), -1.0):            # 0, infinite, infinite, negative as a float
        assert _append(fk, rope=fk.rope_desc(mscale=x)) == fk.FUSE_ERR_INVALID_ARG, x
    assert _append(fk, rope=fk.rope_desc(mscale=1.25), n_rows=0) == fk.FUSE_OK
