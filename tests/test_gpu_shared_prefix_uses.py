"""Shared-prefix attention as servers call it: several queries of one
sequence (speculative tokens, a chunk of a prompt), values that are not
finite, and the size of the error over a whole output."""
import numpy as np
import pytest
import torch

from conftest import cuda_ok
from long_context_decode_indexer_b200 import dsa
from long_context_decode_indexer_b200.batch import workspace
from serving_ref import attention, check_attention

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

SCALE = 576 ** -0.5


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


class Chunks:
    """groups: list of (shared positions, [(cached, new) of each sequence]).
    A sequence's `new` queries see cached + 1, .., cached + new positions."""

    def __init__(self, groups, h, page, seed=0, temp=2.0, pad=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        seqs = [(gi, p, c, n) for gi, (p, ss) in enumerate(groups) for c, n in ss]
        first = {}
        q_seq, q_n, rows_of = [], [], []
        width = max(-(-(c + n) // max(page, 1)) for _, _, c, n in seqs) if page else 0
        table, row0, used = np.full((len(seqs), max(width, 1)), -5), np.zeros(len(seqs), np.int64), 0
        for b, (gi, p, c, n) in enumerate(seqs):
            a = first.setdefault(gi, b)
            pos = np.arange(c + n)
            if page:
                shared = p // page if a != b else 0
                cnt = -(-(c + n) // page)
                table[b, :shared] = table[a, :shared]
                table[b, shared:cnt] = np.arange(used, used + cnt - shared)
                used += cnt - shared
            else:
                row0[b] = used - (p if a != b else 0)
                used += c + n - (p if a != b else 0)
        if page:
            perm = rng.permutation(used)
            table = np.where(table >= 0, perm[table.clip(0)], -5)
        at = (lambda b, s: table[b, s // page] * page + s % page) if page else (lambda b, s: row0[b] + s)
        for b, (gi, p, c, n) in enumerate(seqs):
            a = first[gi]
            full = np.r_[at(a, np.arange(p)), at(b, np.arange(p, c + n))]
            for i in range(n):
                q_seq.append(b)
                q_n.append(c + 1 + i)
                rows_of.append(full[:c + 1 + i])
        q_seq += [0] * pad
        q_n += [0] * pad
        rows_of += [np.zeros(0, np.int64)] * pad
        nq, rows = len(q_n), used * page if page else used
        self.lists = [torch.from_numpy(np.asarray(x, np.int64)).cuda() for x in rows_of]
        self.kv = torch.full((rows, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
        live = torch.unique(torch.cat(self.lists))
        self.kv[live] = torch.randn((len(live), 576), generator=g, device="cuda").bfloat16()
        self.q = (torch.randn((nq, h, 576), generator=g, device="cuda") * temp).bfloat16()
        per = [sum(n for _, n in ss) for _, ss in groups]
        per[-1] += pad
        self.keep = [_i32(q_seq), _i32(q_n), torch.from_numpy(row0).cuda(), _i32(table), _i32(np.r_[0, np.cumsum(per)]),
                     _i32([p for p, _ in groups])]
        self.p = dsa.make_params(nq=nq, h_idx=64, d_idx=128, h=h, topk=1, max_n=max(q_n), q_per_seq=1, scale=SCALE)
        self.kvd = dsa.make_kv(q_seq=self.keep[0], q_n=self.keep[1], seq_row0=None if page else self.keep[2],
                               page_table=self.keep[3] if page else None, page_size=page, cache_rows=rows)
        self.ng = len(groups)
        self.ws = workspace(dsa.shared_prefix_workspace_size(self.p, self.kvd, self.ng))

    def run(self, q=None):
        q = self.q if q is None else q
        out = torch.full((*q.shape[:2], 512), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], 5.0, device="cuda")
        dsa.mla_shared_prefix(self.p, self.kvd, self.ng, self.keep[4], self.keep[5], q, self.kv, 576, out, lse, self.ws)
        assert dsa.check_status(self.ws) == dsa.DSA_OK
        return out, lse

    def ref(self, i):
        rows = self.kv[self.lists[i]].double()
        q = self.q[i].double()
        span = float((q.abs() @ rows.abs().t()).max()) * SCALE if len(rows) else 0.0
        return attention(q, rows, SCALE), span

    def check(self, out, lse, sel):
        for i in sel:
            (ref, rl, mag, rms), span = self.ref(i)
            check_attention(out[i], lse[i], ref, rl, mag, rms, span)


@pytest.mark.parametrize("page", [0, 64, 128])
@pytest.mark.parametrize("h", [1, 16, 128])
@pytest.mark.parametrize("per", [2, 4])
def test_speculative_tokens(page, h, per):
    """Consecutive queries of a sequence, each one position further."""
    c = Chunks([(1000, [(1000, per), (1127, per), (1500, per)]), (0, [(0, per), (63, per), (64, per)]),
                (300, [(299 + per, per)] * 5)], h, page, seed=h + per, pad=3)
    out, lse = c.run()
    c.check(out, lse, range(c.q.shape[0]))


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("h,new,prefix", [(16, 300, 5000), (128, 65, 129), (5, 1024, 0)])
def test_a_chunk_of_a_prompt(page, h, new, prefix):
    """All new tokens of one prompt, causal, behind what is cached; another
    prompt behind the same prefix."""
    c = Chunks([(prefix, [(prefix, new), (prefix + 70, 33)])], h, page, seed=new)
    out, lse = c.run()
    n = c.q.shape[0]
    c.check(out, lse, sorted({0, 1, 62, 63, 64, new // 2, new - 1, new, n - 1} & set(range(n))))


def test_a_prompt_in_chunks_equals_the_prompt_in_one():
    """4096 queries are the most of one call: a longer prompt goes in parts.
    A query's result does not depend on the part it is in, but for the order
    of its sums."""
    whole = Chunks([(0, [(0, 600)])], 16, 64, seed=3)
    out, lse = whole.run()
    sel = [0, 255, 256, 399, 599]
    whole.check(out, lse, sel)
    for lo, hi in ((0, 256), (256, 600)):
        p = dsa.make_params(nq=hi - lo, h_idx=64, d_idx=128, h=16, topk=1, max_n=600, scale=SCALE)
        kv = dsa.make_kv(q_seq=whole.keep[0][lo:hi], q_n=whole.keep[1][lo:hi], page_table=whole.keep[3], page_size=64,
                         cache_rows=whole.kv.shape[0])
        ws = workspace(dsa.shared_prefix_workspace_size(p, kv, 1))
        o, l = torch.zeros_like(out[lo:hi]), torch.zeros_like(lse[lo:hi])
        dsa.mla_shared_prefix(p, kv, 1, _i32([0, hi - lo]), _i32([lo]), whole.q[lo:hi], whole.kv, 576, o, l, ws)
        assert dsa.check_status(ws) == dsa.DSA_OK
        for i in sel:
            if lo <= i < hi:
                (ref, rl, mag, rms), span = whole.ref(i)
                check_attention(o[i - lo], l[i - lo], ref, rl, mag, rms, span)


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_not_finite_spoils_itself_alone(page, value):
    c = Chunks([(400, [(400, 2), (470, 2), (900, 1)]), (0, [(77, 3)])], 24, page, seed=5)
    clean, clean_l = c.run()
    q = c.q.clone()
    hit = [(0, 3), (2, 23), (4, 0), (6, 11)]
    for i, hd in hit:
        q[i, hd, 100] = value
    out, lse = c.run(q)
    keep = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    for i, hd in hit:
        keep[i, hd] = False
        # +-inf times rows of both signs: scores of both infinities, NaN as in the formula
        assert torch.all(torch.isnan(out[i, hd])) and torch.isnan(lse[i, hd])
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_l[keep])


@pytest.mark.parametrize("page", [0, 64])
def test_a_visible_row_that_is_not_finite(page):
    """A NaN that a query sees reaches it, and no query that does not."""
    c = Chunks([(300, [(300, 4)])], 16, page, seed=6)
    clean, clean_l = c.run()
    c.kv[c.lists[3][302]] = float("nan")     # the third new token's own row
    out, lse = c.run()
    assert torch.equal(out[:2], clean[:2]) and torch.equal(lse[:2], clean_l[:2])
    assert torch.all(torch.isnan(out[2:])) and torch.all(torch.isnan(lse[2:]))


@pytest.mark.parametrize("temp", [0.5, 2.0, 6.0])
def test_the_error_of_a_whole_output(temp):
    """The 2-norm of the error against what two roundings to nearest predict:
    the output's (a step^2 / 12 of each value) and every weight's (mantissas
    spread like 1 / m: 2^-14 / 12 * 0.541 of P^2), independent of each other,
    30% more for chance and for mantissas that are spread otherwise.  Weights
    rounded toward zero would lose 2^-8 * 0.72 of the output each: 2.4 times
    the square.  One at a time they could not be told."""
    c = Chunks([(3000, [(3000 + 40 * k, 1) for k in range(12)])], 64, 64, seed=7, temp=temp)
    out, _ = c.run()
    err = want = 0.0
    for i in range(12):
        (ref, _, mag, rms), _ = c.ref(i)
        e = out[i].double() - ref
        step = torch.exp2(torch.floor(torch.log2(ref.abs().clamp(min=1e-30))) - 7)
        err += float((e * e).sum())
        want += float((step * step).sum()) / 12 + 2.0 ** -14 / 12 * 0.541 * float((rms * rms).sum())
    assert err <= 1.3 * want, "square error %.3g of what is predicted" % (err / want)


@pytest.mark.parametrize("page", [0, 64])
def test_groups_without_queries(page):
    """Groups of no queries before, between and behind the others, more
    groups than queries."""
    c = Chunks([(300, [(300, 2)]), (70, [(90, 1), (70, 1)])], 16, page, seed=8)
    clean, clean_l = c.run()
    q0, n = c.keep[4].tolist(), c.keep[5].tolist()
    c.keep[4] = _i32([0, 0, 0, q0[1], q0[1], q0[1], q0[2], q0[2], q0[2]])
    c.keep[5] = _i32([5, 300, n[0], 0, 299, n[1], 64, 1])
    c.ng = 8
    c.ws = workspace(dsa.shared_prefix_workspace_size(c.p, c.kvd, 8))
    out, lse = c.run()
    c.check(out, lse, range(4))
    assert torch.equal(out, clean) and torch.equal(lse, clean_l)
