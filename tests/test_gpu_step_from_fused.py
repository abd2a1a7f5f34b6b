"""From a fused cache to generation: what the fusion writes is read as pages by
the operators of a step, without a copy."""

import math

import numpy as np
import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk, synth

from harness import buffers, make_case, request_slices
from step_ops import DT, HALF_STEP, ancestors, check_close, depths, f64, i32, random_tree, rotate, thetas

pytestmark = pytest.mark.gpu


# A request's fused rows lie one behind the other from its first row on.  A single one's
# are pages of any size, its last page partly filled; packed ones start anywhere, so that
# their pages are single rows.  Pages behind the fused rows take the new tokens.
@pytest.mark.parametrize("dtype,requests,block_size", [("f32", 1, 16), ("bf16", 1, 64), ("bf16", 3, 1), ("f32", 2, 1)])
def test_tokens_behind_a_fused_cache(dtype, requests, block_size):
    cfg = synth.scaled(synth.CONFIGS["tiny_fp32"], dtype=dtype, kv_storage=dtype, n_requests=requests, query_len=9)
    case = make_case(cfg)
    b = buffers(case)
    Hq, Hkv, d = cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim
    parts = [(row0, T) for _, row0, _, T, _ in request_slices(case)]
    total = parts[-1][0] + parts[-1][1]
    rng = np.random.default_rng(block_size)
    new = [int(x) for x in rng.integers(5, 20, requests)]
    # pools with room behind the fused rows; the fusion writes into their front
    spare = [-(-(n + block_size) // block_size) for n in new]
    pages = -(-total // block_size) + sum(spare)
    dt = DT[dtype]
    kp, vp = (torch.zeros(pages, block_size, Hkv, d, dtype=dt, device="cuda") for _ in range(2))
    Kf, Vf = kp.view(-1, Hkv, d), vp.view(-1, Hkv, d)
    fk.layer_step(b.desc, b.chunks, b.reqs, b.H, b.Wq, b.Wk, b.Wv, True, b.idx, Kf, Vf, b.O, b.score, b.ws)
    fk.check_errors(b.ws)
    kf, vf = f64(Kf)[:total], f64(Vf)[:total]
    assert np.abs(kf).max(-1).all() and np.abs(vf).max(-1).all()
    tables, at = [], -(-total // block_size)
    for (row0, T), k in zip(parts, spare):
        tables.append([row0 // block_size + i for i in range(-(-T // block_size))] + [at + i for i in range(k)])
        at += k
    tab = np.full((requests, max(map(len, tables))), -1, np.int32)
    for row, t in zip(tab, tables):
        row[:len(t)] = t
    starts = [sum(new[:i]) for i in range(requests + 1)]
    trees = [random_tree(n, 3, rng) for n in new]
    lens = i32([T for _, T in parts])
    seqs = fk.Sequences(i32(tab), lens, i32(starts), block_size, pages, max(new))
    parents = i32([p for t in trees for p in t])
    qkv = torch.from_numpy(rng.standard_normal((starts[-1], Hq + 2 * Hkv, d)).astype(np.float32)).to(dt).cuda()
    Q, K, V = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    Qr, O = torch.zeros(starts[-1], Hq, d, dtype=dt, device="cuda"), torch.zeros(starts[-1], Hq, d, dtype=dt, device="cuda")
    ws = fk.alloc_tree_workspace(b.desc, seqs)
    fk.cache_append(b.desc, fk.rope_desc(), seqs, parents, Q, K, V, Qr, None, kp, vp, ws)
    fk.attend_tree(b.desc, seqs, parents, Qr, kp, vp, O, ws)
    fk.check_errors(ws)
    assert np.array_equal(f64(Kf)[:total], kf) and np.array_equal(f64(Vf)[:total], vf)
    theta, x = thetas(cfg.rope_base, d), f64(qkv)
    for r, (row0, T) in enumerate(parts):
        a, e = starts[r], starts[r + 1]
        # new rows turn at the positions behind the request's own
        y, tol = rotate(x[a:e, :Hq + Hkv], T + np.array(depths(trees[r])), theta, fk.FUSE_ROPE_HALF, 1.0, dtype)
        check_close(f64(Qr)[a:e], y[:, :Hq], tol[:, :Hq], "Qr")
        slot = T + np.arange(new[r])
        kn = f64(kp)[tab[r, slot // block_size], slot % block_size]
        check_close(kn, y[:, Hq:], tol[:, Hq:], "new keys")
        keys = np.concatenate([kf[row0:row0 + T], kn])
        values = np.concatenate([vf[row0:row0 + T], x[a:e, Hq + Hkv:]])
        seen = np.concatenate([np.ones((new[r], T), bool), ancestors(trees[r])], 1)
        q, got = f64(Qr)[a:e], f64(O)[a:e]
        for i in range(new[r]):
            for h in range(Hq):
                k, v = keys[seen[i], h * Hkv // Hq], values[seen[i], h * Hkv // Hq]
                z = k @ q[i, h] / math.sqrt(d)
                p = np.exp(z - z.max())
                p /= p.sum()
                # as step_ops.Step.tree_reference
                S = np.max(np.abs(k) @ np.abs(q[i, h])) / math.sqrt(d)
                err = S * ((d + 16) * 2.0 ** -23 + 2.0 ** -21)
                w = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -21
                bound = HALF_STEP[dtype] * np.abs(p @ v) + (w + 2 * err + len(k) * 2.0 ** -24) * (p @ np.abs(v))
                assert np.all(np.abs(got[i, h] - p @ v) <= bound)
