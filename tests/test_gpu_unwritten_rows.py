"""Sparse attention over a cache whose rows nobody has written hold NaN or
infinities: empty entries of the index list (-1, behind the list's end, a
position not visible) must not bring any of it into the output."""
import numpy as np
import pytest
import torch

from conftest import cuda_ok
from long_context_decode_indexer_b200 import dsa
from long_context_decode_indexer_b200.batch import workspace
from serving_ref import attention

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

SCALE = 576 ** -0.5


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _run(fp8, prefill, h, topk, counts, page, fill, seed):
    """Queries with `counts[i]` entries at random places of their lists, the
    selected rows written and everything else `fill` or zero."""
    rng = np.random.default_rng(seed)
    nq, n, rows = len(counts), 700, 1024
    table = np.stack([rng.permutation(np.arange(1, rows // 64))[:11] for _ in range(nq)])   # nobody has page 0
    idx = np.full((nq, topk), -1, np.int64)
    want = []
    for i, c in enumerate(counts):
        pos = rng.permutation(n)[:c]
        idx[i, rng.permutation(topk)[:c]] = pos
        want.append(table[i, pos // 64] * 64 + pos % 64 if page else 64 + pos)
    used = np.zeros(rows, bool)
    for w in want:
        used[w] = True
    used = torch.from_numpy(used).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randn((nq, h, 576), generator=g, device="cuda").bfloat16()
    live = torch.randn((rows, 576), generator=g, device="cuda")
    p = dsa.make_params(nq=nq, h_idx=4, d_idx=128, h=h, topk=topk, max_n=704, scale=SCALE)
    row0 = torch.full((nq,), 64, dtype=torch.int64, device="cuda")
    q_seq, q_n, tab = _i32(np.arange(nq)), _i32(np.full(nq, n)), _i32(table)
    kv = dsa.make_kv(q_seq=q_seq, q_n=q_n, seq_row0=None if page else row0, page_table=tab if page else None,
                     page_size=page, cache_rows=rows)
    ws = workspace(dsa.workspace_size(p, kv, dsa.OP_SPARSE_MLA_DECODE))
    ix = _i32(idx)
    got = []
    for bad in (0.0, fill):
        out = torch.full((nq, h, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((nq, h), 5.0, device="cuda")
        if fp8:
            c = live.to(torch.float8_e4m3fn).view(torch.uint8).clone()
            sc = torch.full((rows,), 0.5, device="cuda")
            c[~used] = 0 if bad == 0 else 0x7F      # the code of NaN
            sc[~used] = bad
            dsa.sparse_mla_decode_fp8(p, kv, q, c, 576, sc, ix, out, lse, ws)
            values = c.view(torch.float8_e4m3fn).double() * sc.double()[:, None]
        else:
            c = live.bfloat16()
            c[~used] = bad
            (dsa.sparse_mla_prefill if prefill else dsa.sparse_mla_decode)(p, kv, q, c, 576, ix, out, lse, ws)
            values = c.double()
        assert dsa.check_status(ws) == dsa.DSA_OK
        got.append((out, lse))
    # bit by bit what a cache with zeros there gives
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16))
    assert torch.equal(got[0][1].view(torch.int32), got[1][1].view(torch.int32))
    out, lse = got[1]
    for i, w in enumerate(want):
        ref, rl, mag, _ = attention(q[i].double(), values[torch.from_numpy(w).cuda()], SCALE)
        if not len(w):
            assert not out[i].any() and torch.all(torch.isneginf(lse[i]))
            continue
        # bf16 output, fp16 split partials (2^-11 of the half row's largest
        # value), 2^-13 of the magnitudes for P as a bf16 pair and fp32 sums
        err = (out[i].double() - ref).abs()
        assert torch.all(err <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * ref.abs().amax() + 2.0 ** -13 * mag)
        assert float((lse[i].double() - rl).abs().max()) <= 1e-3


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("kind", ["bf16", "prefill", "fp8"])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("h,topk,counts", [
    (128, 256, [256, 255, 1, 0]), (16, 100, [99, 0, 17, 100, 33]), (5, 7, [1, 0, 6]),
    (16, 2048, [3, 700, 0]),                        # splits with no valid entry
    (64, 512, [500] * 160)])                        # one split a query
def test_unwritten_rows_stay_out(page, kind, fill, h, topk, counts):
    _run(kind == "fp8", kind == "prefill", h, topk, counts, page, fill, seed=topk + len(counts))


def test_entries_that_are_not_visible_stay_out():
    """An entry at or past q_n is flagged and skipped, whatever row 0 holds."""
    nq, h, topk = 2, 8, 64
    kv_c = torch.randn((200, 576), device="cuda").bfloat16()
    kv_c[0] = float("nan")
    q = torch.randn((nq, h, 576), device="cuda").bfloat16()
    idx = _i32(np.stack([np.r_[np.arange(40), [100, 150], np.full(22, -1)], np.full(64, 100)]))
    p = dsa.make_params(nq=nq, h_idx=4, d_idx=128, h=h, topk=topk, max_n=128, scale=SCALE)
    row0, q_seq, q_n = torch.full((1,), 1, dtype=torch.int64, device="cuda"), _i32([0, 0]), _i32([100, 100])
    kv = dsa.make_kv(q_seq=q_seq, q_n=q_n, seq_row0=row0, cache_rows=200)
    ws = workspace(dsa.workspace_size(p, kv, dsa.OP_SPARSE_MLA_DECODE))
    out, lse = torch.zeros((nq, h, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((nq, h), device="cuda")
    dsa.sparse_mla_decode(p, kv, q, kv_c, 576, idx, out, lse, ws)
    assert dsa.check_status(ws) == dsa.DSA_ERR_DEVICE_CHECK
    ref, rl, mag, _ = attention(q[0].double(), kv_c[1:41].double(), SCALE)
    assert torch.all((out[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * ref.abs().amax() + 2.0 ** -13 * mag)
    assert not out[1].any() and torch.all(torch.isneginf(lse[1]))


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("d_qk,d_v", [(192, 128), (64, 64)])
@pytest.mark.parametrize("lengths", [[1], [100, 128, 129], [300], [16, 383]])
def test_masked_mha_of_rows_behind_the_sequences(fill, d_qk, d_v, lengths):
    """Sequences of one length each, apart in k and v; the rows between and
    behind them are nobody's."""
    L, h, gap = max(lengths), 3, 200
    nq, rows = L * len(lengths), (L + gap) * len(lengths)
    g = torch.Generator(device="cuda")
    g.manual_seed(L)
    q = torch.randn((nq, h, d_qk), generator=g, device="cuda").bfloat16()
    k, v = (torch.randn((rows, h, d), generator=g, device="cuda").bfloat16() for d in (d_qk, d_v))
    row0 = np.arange(len(lengths)) * (L + gap)
    n = np.concatenate([np.minimum(np.arange(1, L + 1), x) for x in lengths])
    used = np.zeros(rows, bool)
    for r, x in zip(row0, lengths):
        used[r:r + x] = True
    used = torch.from_numpy(used).cuda()
    p = dsa.make_params(nq=nq, h_idx=1, d_idx=64, h=h, topk=1, max_n=L, q_per_seq=L, scale=d_qk ** -0.5, d_qk=d_qk, d_v=d_v)
    keep = [_i32(np.repeat(np.arange(len(lengths)), L)), _i32(n), torch.from_numpy(row0).cuda()]
    kv = dsa.make_kv(q_seq=keep[0], q_n=keep[1], seq_row0=keep[2], cache_rows=rows)
    ws = workspace(dsa.workspace_size(p, kv, dsa.OP_MASKED_MHA))
    got = []
    for bad in (0.0, fill):
        k[~used], v[~used] = bad, bad
        out = torch.full((nq, h, d_v), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((nq, h), 5.0, device="cuda")
        dsa.masked_mha_prefill(p, kv, q, k, v, None, out, lse, ws)
        assert dsa.check_status(ws) == dsa.DSA_OK
        got.append((out, lse))
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])
    for t in (0, L - 1, nq - 1):
        b, m = t // L, int(n[t])
        kk, vv = (x[row0[b]:row0[b] + m].double().transpose(0, 1) for x in (k, v))
        s = torch.einsum("hd,hsd->hs", q[t].double(), kk) * d_qk ** -0.5
        ref = torch.einsum("hs,hsd->hd", torch.softmax(s, 1), vv)
        mag = torch.einsum("hs,hsd->hd", torch.softmax(s, 1), vv.abs())
        # bf16 output; P as a bf16 pair and fp32 sums 2^-13 of the magnitudes
        assert torch.all((got[1][0][t].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * mag)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_served_cache_that_was_never_cleared(fp8):
    """Tables, append and sparse attention over a cache that starts as NaN:
    page 0 is never handed out, the lists are longer than the histories."""
    rng = np.random.default_rng(0)
    nseq, h, topk, rows = 3, 16, 256, 12 * 64
    new = np.array([100, 1, 64])
    nt = int(new.sum()) + 4
    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    seq, head, table = z(nseq), z(1), _i32(np.full((nseq, 4), -1))
    q_start, q_seq, pos, q_n, slots = z(nseq + 1), z(nt), z(nt), z(nt), z(nt)
    tp = dsa.make_table_params(nseq=nseq, nt=nt, page_size=64, max_pages=4, n_free=11, cache_rows=rows)
    ws = workspace(dsa.table_workspace_size(tp))
    dsa.build_tables(tp, seq, _i32(new), None, _i32(rng.permutation(np.arange(1, 12))), head, table, q_start, q_seq, pos,
                     q_n, slots, seq, head, ws)
    kv_a = torch.from_numpy(rng.standard_normal((nt, 576))).bfloat16().cuda()
    rs = dsa.make_rope_spec()
    if fp8:
        cache = torch.full((rows, 576), 0x7F, dtype=torch.uint8, device="cuda")
        sc = torch.full((rows,), float("nan"), device="cuda")
        dsa.latent_append_fp8(rs, kv_a[:, :512], kv_a[:, 512:], pos, slots, cache, sc, ws)
        values = cache.view(torch.float8_e4m3fn).double() * sc.double()[:, None]
    else:
        cache = torch.full((rows, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
        dsa.latent_append(rs, kv_a[:, :512], kv_a[:, 512:], pos, slots, cache, ws)
        values = cache.double()
    idx = np.full((nseq, topk), -1)
    for b in range(nseq):
        idx[b, :new[b]] = np.arange(new[b])
    last = (q_start[1:] - 1).long()
    q = torch.from_numpy(rng.standard_normal((nseq, h, 576))).bfloat16().cuda()
    qs, qn = q_seq[last].contiguous(), q_n[last].contiguous()
    p = dsa.make_params(nq=nseq, h_idx=4, d_idx=128, h=h, topk=topk, max_n=256, scale=SCALE)
    kv = dsa.make_kv(q_seq=qs, q_n=qn, page_table=table, page_size=64, cache_rows=rows)
    ws_m = workspace(dsa.workspace_size(p, kv, dsa.OP_SPARSE_MLA_DECODE))
    out, lse = torch.zeros((nseq, h, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((nseq, h), device="cuda")
    if fp8:
        dsa.sparse_mla_decode_fp8(p, kv, q, cache, 576, sc, _i32(idx), out, lse, ws_m)
    else:
        dsa.sparse_mla_decode(p, kv, q, cache, 576, _i32(idx), out, lse, ws_m)
    assert dsa.check_status(ws) == dsa.check_status(ws_m) == dsa.DSA_OK
    for b in range(nseq):
        at = slots[int(q_start[b]):int(q_start[b + 1])].long()
        ref, rl, mag, _ = attention(q[b].double(), values[at], SCALE)
        err = (out[b].double() - ref).abs()
        assert torch.all(err <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * ref.abs().amax() + 2.0 ** -13 * mag)
        assert float((lse[b].double() - rl).abs().max()) <= 1e-3
