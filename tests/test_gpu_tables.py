"""Page tables and slot maps built on the GPU, against a plain loop: every
number has to be equal."""
import numpy as np
import pytest
import torch

from conftest import cuda_ok
from long_context_decode_indexer_b200 import dsa
from long_context_decode_indexer_b200.batch import workspace
from serving_ref import tables as ref_tables

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

FILL = -77
OUT = ("q_start", "q_seq", "pos", "q_n", "slots", "kv_len", "head")


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


class Step:
    """One call's device arrays, outputs behind a guard."""

    def __init__(self, seq, new, free, table, nt, ps, n_pages, fork=None, head=0, sees_self=1, alias=False):
        n = len(seq)
        self.host = dict(seq=seq, new=new, fork=fork, free=free, head=head, table=table, nt=nt, ps=ps,
                         n_pages=n_pages, sees_self=sees_self)
        self.tp = dsa.make_table_params(nseq=n, nt=nt, page_size=ps, max_pages=table.shape[1], n_free=len(free),
                                        cache_rows=n_pages * ps + ps // 2, sees_self=sees_self)
        self.seq, self.new = _i32(seq), _i32(new)
        self.fork = None if fork is None else _i32(fork)
        self.free, self.head_in, self.table = _i32(free), _i32([head]), _i32(table)
        size = dict(q_start=n + 1, q_seq=nt, pos=nt, q_n=nt, slots=nt, kv_len=n, head=1)
        self.buf = {k: torch.full((v + 64,), FILL, dtype=torch.int32, device="cuda") for k, v in size.items()}
        self.out = {k: self.buf[k][:v] for k, v in size.items()}
        if alias:
            self.out["kv_len"], self.out["head"] = self.seq, self.head_in
        self.ws = workspace(dsa.table_workspace_size(self.tp))

    def call(self):
        o = self.out
        dsa.build_tables(self.tp, self.seq, self.new, self.fork, self.free, self.head_in, self.table, o["q_start"],
                         o["q_seq"], o["pos"], o["q_n"], o["slots"], o["kv_len"], o["head"], self.ws)

    def check(self):
        """Equal to the loop, or refused as the loop refuses it."""
        h = self.host
        ref = ref_tables(h["seq"], h["new"], h["fork"], h["free"], h["head"], h["table"], h["nt"], h["ps"],
                         h["n_pages"], h["sees_self"])
        got = {k: v.cpu().numpy() for k, v in self.out.items()}
        for k in OUT:
            assert np.all(self.buf[k].cpu().numpy()[len(self.out[k]):] == FILL), k
        status = dsa.check_status(self.ws)
        if ref is None:
            assert status == dsa.DSA_ERR_DEVICE_CHECK
            assert np.array_equal(self.table.cpu().numpy(), h["table"])
            assert got["head"][0] == h["head"] and np.array_equal(got["kv_len"], h["seq"])
            assert not got["q_start"].any() and not got["q_seq"].any() and not got["q_n"].any()
            assert np.all(got["pos"] == -1) and np.all(got["slots"] == -1)
            return
        assert status == (dsa.DSA_ERR_DEVICE_CHECK if ref["bad"] else dsa.DSA_OK)
        assert np.array_equal(self.table.cpu().numpy(), ref["table"])
        for k in OUT:
            assert np.array_equal(got[k].reshape(-1), np.ravel(ref[k])), k
        return ref


def _batch(rng, n, ps, top, forks=0, prefill=0):
    seq = rng.integers(0, top, n)
    new = rng.integers(0, 4, n)
    if prefill:
        new[rng.integers(0, n, 3)] = prefill
    fork = np.full(n, -1)
    if forks:
        kids = rng.permutation(n)[:forks]
        parents = np.setdiff1d(np.arange(n), kids)
        for b in kids:
            fork[b] = rng.choice(parents)
            seq[b] = rng.integers(0, seq[fork[b]] // ps + 1) * ps
    held = -(-seq // ps)
    pages = held.copy()
    pages[fork >= 0] = 0
    need = (-(-(seq + new) // ps) - held).sum()
    n_pages = int(pages.sum() + need + 5)
    perm = rng.permutation(n_pages)
    table = np.full((n, int((-(-(seq + new) // ps)).max()) + 2), FILL)
    at = 0
    for b in range(n):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
    return seq, new, (fork if forks else None), perm[at:], table, n_pages


@pytest.mark.parametrize("n,ps,top,forks,prefill,pad", [
    (1, 64, 1, 0, 0, 0), (1, 64, 200, 0, 5000, 1), (2, 1, 9, 0, 0, 3), (7, 7, 100, 2, 40, 0),
    (128, 64, 40000, 0, 0, 0), (129, 128, 3000, 30, 700, 17), (600, 64, 2000, 40, 3000, 1000),
    (4096, 64, 700, 200, 0, 5), (16384, 16, 60, 0, 33, 1)])
@pytest.mark.parametrize("sees_self", [0, 1])
def test_tables_equal_the_loop(n, ps, top, forks, prefill, pad, sees_self):
    rng = np.random.default_rng(n + ps)
    seq, new, fork, free, table, n_pages = _batch(rng, n, ps, top, forks, prefill)
    free = np.r_[[0, 0, 0], free]
    s = Step(seq, new, free, table, int(new.sum()) + pad, ps, n_pages, fork=fork, head=3, sees_self=sees_self)
    s.call()
    assert s.check() is not None
    s.call()                    # the same call again gives the same tables
    s.check()


def test_token_arrays_at_odd_addresses():
    rng = np.random.default_rng(3)
    seq, new, fork, free, table, n_pages = _batch(rng, 50, 64, 500, 5, 333)
    nt = int(new.sum()) + 3
    s = Step(seq, new, free, table, nt, 64, n_pages, fork=fork)
    for k, off in (("q_seq", 1), ("pos", 2), ("q_n", 3), ("slots", 1)):
        s.buf[k] = torch.full((nt + 68,), FILL, dtype=torch.int32, device="cuda")[off:]
        s.out[k] = s.buf[k][:nt]
    s.call()
    assert s.check() is not None


def test_no_sequences_and_no_tokens():
    s = Step(np.zeros(0, int), np.zeros(0, int), np.arange(2), np.zeros((0, 3), int), 5, 64, 4)
    s.call()
    s.check()
    s = Step(np.array([64, 63, 0]), np.zeros(3, int), np.arange(2), np.full((3, 2), 1), 0, 64, 4)
    s.call()
    s.check()


def test_every_page_is_used_and_lengths_end_at_the_limit():
    """The last free page, a table filled to its last entry, page borders."""
    seq, new = np.array([63, 64, 65, 0, 128]), np.array([1, 1, 127, 192, 64])
    table = np.full((5, 3), FILL)
    table[0, 0], table[1, 0], table[2, :2], table[4, :2] = 9, 8, (7, 6), (5, 4)
    s = Step(seq, new, np.array([0, 1, 2, 3, 10, 11]), table, int(new.sum()), 64, 12)
    s.call()
    assert s.check()["head"] == 6


@pytest.mark.parametrize("kind", ["negative", "negative_new", "long", "tokens", "pages", "head", "head_past_end",
                                  "fork_range", "fork_self", "fork_of_fork", "fork_part_page", "fork_long",
                                  "overflow"])
def test_a_batch_that_cannot_be_laid_out_changes_nothing(kind):
    seq, new = np.array([100, 64, 0, 128]), np.array([1, 1, 70, 2])
    table = np.full((4, 4), FILL)
    table[0, :2], table[1, 0], table[3, :2] = (0, 1), 2, (3, 4)
    fork, nt, head, free = None, 80, 0, np.arange(5, 12)
    if kind == "negative": seq[1] = -1
    if kind == "negative_new": new[2] = -3
    if kind == "long": new[0], nt = 157, 1000
    if kind == "tokens": nt = 73
    if kind == "pages": free = free[:3]
    if kind == "head": head = -1
    if kind == "head_past_end": head = 8
    if kind == "overflow": new[0], new[1] = 2 ** 31 - 1, 2 ** 31 - 1
    if kind.startswith("fork"):
        fork = np.full(4, -1)
        fork[2] = {"fork_range": 4, "fork_self": 2}.get(kind, 3)
        if kind == "fork_of_fork": fork[3] = 0
        if kind == "fork_part_page": seq[2] = 65
        if kind == "fork_long": seq[2] = 192
    s = Step(seq, new, free, table, nt, 64, 12, fork=fork, head=head)
    s.call()
    assert s.check() is None
    # the workspace serves the next call
    s.ws2 = s.ws
    ok = Step(np.array([100]), np.array([1]), np.arange(4), np.array([[0, 1]]), 1, 64, 8)
    ok.ws = s.ws
    ok.call()
    ok.check()


def test_page_ids_outside_the_cache_are_flagged():
    """A bad new page and a bad entry of the table: slots of -1, a flag, the
    rest laid out."""
    table = np.array([[0, 99, FILL], [1, FILL, FILL], [2, FILL, FILL]])
    s = Step(np.array([100, 64, 10]), np.array([5, 3, 2]), np.array([-4, 6]), table, 12, 64, 8)
    s.call()
    assert s.check()["bad"]


def test_lengths_and_head_advance_in_place_through_a_captured_step():
    """kv_len is seq_len and the new head is the head: a captured call laid
    out again and again gives one sequence of tables."""
    rng = np.random.default_rng(0)
    n, ps, steps = 150, 64, 70
    seq = rng.integers(0, 300, n)
    new = rng.integers(0, 3, n)
    held = -(-seq // ps)
    n_pages = int(held.sum()) + n * 6
    perm = rng.permutation(n_pages)
    table = np.full((n, 12), FILL)
    at = 0
    for b in range(n):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    s = Step(seq, new, perm[at:], table, int(new.sum()) + 4, ps, n_pages, alias=True)
    keep = (s.seq.clone(), s.table.clone(), s.head_in.clone())
    s.call()
    for dst, src in zip((s.seq, s.table, s.head_in), keep):
        dst.copy_(src)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call()
    for _ in range(steps):
        g.replay()
        torch.cuda.synchronize()
        ref = ref_tables(seq, new, None, perm[at:], s.host["head"], table, s.tp.nt, ps, n_pages, 1)
        assert np.array_equal(s.seq.cpu().numpy(), ref["kv_len"])
        assert int(s.head_in) == ref["head"]
        assert np.array_equal(s.table.cpu().numpy(), ref["table"])
        for k in ("q_start", "q_seq", "pos", "q_n", "slots"):
            assert np.array_equal(s.out[k].cpu().numpy(), ref[k]), k
        seq, table, s.host["head"] = ref["kv_len"], ref["table"], ref["head"]
    assert dsa.check_status(s.ws) == dsa.DSA_OK


def test_calls_on_two_streams():
    rng = np.random.default_rng(5)
    steps = []
    for k in range(4):
        seq, new, fork, free, table, n_pages = _batch(rng, 300, 64, 500, 20, 200)
        steps.append(Step(seq, new, free, table, int(new.sum()), 64, n_pages, fork=fork))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k, s in enumerate(steps):
        with torch.cuda.stream(streams[k % 2]):
            s.call()
    torch.cuda.synchronize()
    for s in steps:
        s.check()


@pytest.mark.parametrize("alias", ["both", "lengths", "head"])
@pytest.mark.parametrize("fill", [0xAB, 1])
def test_in_place_on_a_workspace_that_another_call_wrote(alias, fill):
    """Only the status word of a workspace has to hold from call to call:
    lengths and head advance in place whatever the rest of it holds."""
    rng = np.random.default_rng(8)
    seq, new, fork, free, table, n_pages = _batch(rng, 600, 64, 2000, 0, 3000)
    s = Step(seq, new, free, table, int(new.sum()) + 3, 64, n_pages)
    if alias != "head":
        s.out["kv_len"] = s.seq
    if alias != "lengths":
        s.out["head"] = s.head_in
    s.ws[dsa.WS_STATUS_BYTES:] = fill
    s.call()
    assert s.check() is not None
    # a refused batch keeps both
    s2 = Step(seq, new, free, table, int(new.sum()) - 1, 64, n_pages, alias=True)
    s2.ws = s.ws
    s2.ws[dsa.WS_STATUS_BYTES:] = fill
    s2.call()
    assert s2.check() is None


@pytest.mark.parametrize("n", [1, 60, 65, 130, 200, 300, 500, 512, 513, 2000])
def test_in_place_at_every_grid(n):
    """One CTA, clusters of up to eight, more than eight."""
    rng = np.random.default_rng(n)
    seq, new, fork, free, table, n_pages = _batch(rng, n, 64, 300, 0, 40)
    s = Step(seq, new, free, table, int(new.sum()) + 1, 64, n_pages, alias=True)
    s.ws[dsa.WS_STATUS_BYTES:] = 0x55
    s.call()
    assert s.check() is not None
    s2 = Step(seq, new, free[:0], table, int(new.sum()) + 1, 64, n_pages, alias=True)   # no page to give
    if (-(-(seq + new) // 64)).sum() > (-(-seq // 64)).sum():
        s2.call()
        assert s2.check() is None
