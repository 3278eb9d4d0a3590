"""Host-side checks of the serving operators' C ABI (no GPU needed): what the
documentation rules out is refused before anything is launched."""
import ctypes

import pytest
import torch

from long_context_decode_indexer_b200 import build as dsa_build
from long_context_decode_indexer_b200 import dsa

FAKE = 1 << 40   # an aligned address that no refused call touches
BIG = 1 << 40    # workspace bytes


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


def tables(L, tp, ws=FAKE, ws_bytes=BIG, drop=()):
    names = ("seq_len", "new_len", "fork_src", "free_pages", "free_head", "page_table", "q_start", "q_seq",
             "positions", "q_n", "slots", "kv_len", "free_head_out")
    return L.dsa_build_tables(ctypes.byref(tp), *[None if n in drop else FAKE for n in names], ws, ws_bytes, None)


def tab(**kw):
    base = dict(nseq=4, nt=8, page_size=64, max_pages=10, n_free=5, cache_rows=6400)
    base.update(kw)
    return dsa.make_table_params(**base)


@pytest.mark.parametrize("kw", [dict(nseq=-1), dict(nseq=16385), dict(nt=-1), dict(page_size=0),
                                dict(page_size=65537), dict(max_pages=0), dict(max_pages=1 << 25), dict(n_free=-1),
                                dict(sees_self=2), dict(cache_rows=0), dict(cache_rows=1 << 31)])
def test_table_shapes_are_refused(L, kw):
    assert tables(L, tab(**kw)) == dsa.DSA_ERR_INVALID_ARG
    with pytest.raises(dsa.DsaError):
        dsa.table_workspace_size(tab(**kw))


@pytest.mark.parametrize("name", ["seq_len", "new_len", "free_pages", "free_head", "page_table", "q_start", "q_seq",
                                  "positions", "q_n", "slots", "kv_len", "free_head_out"])
def test_table_null_pointers_are_refused(L, name):
    assert tables(L, tab(), drop=(name,)) == dsa.DSA_ERR_INVALID_ARG


def test_table_workspace_is_checked(L):
    need = dsa.table_workspace_size(tab())
    assert tables(L, tab(), ws=None) == dsa.DSA_ERR_WORKSPACE
    assert tables(L, tab(), ws=FAKE + 64) == dsa.DSA_ERR_WORKSPACE
    assert tables(L, tab(), ws_bytes=need - 1) == dsa.DSA_ERR_WORKSPACE


def rope(L, spec_kw=None, par_kw=None, x=FAKE, y=FAKE + (1 << 30), pos=FAKE, fn="dsa_rope"):
    spec = dsa.make_rope_spec(**(spec_kw or {}))
    base = dict(nt=4, h=8, d=64, dtype=dsa.DTYPE_BF16)
    base.update(par_kw or {})
    return getattr(L, fn)(ctypes.byref(spec), ctypes.byref(dsa.make_rope_params(**base)), x, pos, y, None)


@pytest.mark.parametrize("fn", ["dsa_rope", "dsa_rope_backward"])
@pytest.mark.parametrize("spec", [dict(rope_dim=63), dict(rope_dim=-2), dict(rope_dim=258), dict(layout=2),
                                  dict(scaling=4), dict(theta=0.0), dict(theta=float("nan")),
                                  dict(mscale=float("inf")), dict(scaling=1, factor=0.0),
                                  dict(scaling=2, factor=float("nan")),
                                  dict(scaling=3, factor=4.0, orig_max_pos=0),
                                  dict(scaling=3, factor=4.0, orig_max_pos=10, beta_fast=1.0, beta_slow=2.0),
                                  dict(scaling=3, factor=4.0, orig_max_pos=10, theta=1.0)])
def test_rope_specs_are_refused(L, fn, spec):
    assert rope(L, spec, fn=fn) == dsa.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("par", [dict(nt=-1), dict(h=0), dict(h=65536), dict(x_heads=2), dict(d=32), dict(d=1025),
                                 dict(begin=1), dict(begin=-1), dict(dtype=3), dict(x_strides=(-512, 64)),
                                 dict(y_strides=(512, 32)), dict(y_strides=(32, 64)),
                                 dict(y_strides=(64, 64)), dict(y_strides=(511, 64)), dict(y_strides=(64, 255))])
def test_rope_shapes_are_refused(L, par):
    assert rope(L, par_kw=par) == dsa.DSA_ERR_INVALID_ARG


def test_rope_pointers_are_refused(L):
    assert rope(L, x=None) == dsa.DSA_ERR_INVALID_ARG
    assert rope(L, y=None) == dsa.DSA_ERR_INVALID_ARG
    assert rope(L, pos=None) == dsa.DSA_ERR_INVALID_ARG
    assert rope(L, x=FAKE + 1) == dsa.DSA_ERR_INVALID_ARG
    assert rope(L, par_kw=dict(x_heads=1), y=FAKE) == dsa.DSA_ERR_INVALID_ARG                # in place, broadcast
    assert rope(L, par_kw=dict(y_strides=(1024, 64)), y=FAKE) == dsa.DSA_ERR_INVALID_ARG     # in place, other strides
    assert rope(L, par_kw=dict(nt=1, y_strides=(0, 64)), x=FAKE + 1) == dsa.DSA_ERR_INVALID_ARG   # one token: only x is bad
    # the gradient of a shared head is written once, its source read with y's strides
    assert rope(L, par_kw=dict(x_heads=1, x_strides=(32, 64)), fn="dsa_rope_backward") == dsa.DSA_ERR_INVALID_ARG


def append(L, spec=None, nt=4, c=FAKE, cs=512, pe=FAKE, ps=64, pos=FAKE, slots=FAKE, cache=FAKE, stride=576,
           scale=FAKE, rows=100, ws=FAKE, ws_bytes=256, fp8=False):
    rs = dsa.make_rope_spec(**(spec or {}))
    if fp8:
        return L.dsa_latent_append_fp8(ctypes.byref(rs), nt, c, cs, pe, ps, pos, slots, cache, stride, scale, rows,
                                       ws, ws_bytes, None)
    return L.dsa_latent_append(ctypes.byref(rs), nt, c, cs, pe, ps, pos, slots, cache, stride, rows, ws, ws_bytes,
                               None)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_arguments_are_refused(L, fp8):
    bad = dsa.DSA_ERR_INVALID_ARG
    assert append(L, dict(rope_dim=32), fp8=fp8) == dsa.DSA_ERR_UNSUPPORTED
    for kw in (dict(nt=-1), dict(c=None), dict(c=FAKE + 8), dict(cs=511), dict(cs=516), dict(pe=None),
               dict(pe=FAKE + 4), dict(ps=56), dict(ps=68), dict(pos=None), dict(slots=None), dict(cache=None),
               dict(cache=FAKE + 8), dict(stride=568), dict(stride=580), dict(rows=0), dict(rows=1 << 31)):
        assert append(L, fp8=fp8, **kw) == bad, kw
    if fp8:
        assert append(L, fp8=True, scale=None) == bad
        assert append(L, fp8=True, stride=584) == bad     # 16-byte rows
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(ws_bytes=255)):
        assert append(L, fp8=fp8, **kw) == dsa.DSA_ERR_WORKSPACE


def prefix(L, p=None, kv=None, ng=1, gq=FAKE, gn=FAKE, q=FAKE, c=FAKE, stride=576, out=FAKE, lse=FAKE, ws=FAKE,
           ws_bytes=BIG):
    p = par() if p is None else p
    kv = kvd() if kv is None else kv
    return L.dsa_mla_shared_prefix(ctypes.byref(p), ctypes.byref(kv), ng, gq, gn, q, c, stride, out, lse, ws,
                                   ws_bytes, None)


def par(**kw):
    base = dict(nq=8, h_idx=64, d_idx=128, h=16, topk=1, max_n=4096, scale=0.04)
    base.update(kw)
    return dsa.make_params(**base)


def kvd(**kw):
    base = dict(q_seq=FAKE, q_n=FAKE, seq_row0=FAKE, cache_rows=1 << 20)
    base.update(kw)
    return dsa.make_kv(**base)


def test_shared_prefix_arguments_are_refused(L):
    bad = dsa.DSA_ERR_INVALID_ARG
    for kw in (dict(nq=-1), dict(h=0), dict(h=129), dict(max_n=-1), dict(scale=float("nan"))):
        assert prefix(L, p=par(**kw)) == bad, kw
        with pytest.raises(dsa.DsaError):
            dsa.shared_prefix_workspace_size(par(**kw), kvd(), 1)
    assert prefix(L, p=par(nq=4097)) == dsa.DSA_ERR_UNSUPPORTED
    assert prefix(L, p=par(d_qk=512)) == dsa.DSA_ERR_UNSUPPORTED
    assert prefix(L, kv=kvd(seq_row0=None)) == bad
    for kw in (dict(ng=0), dict(ng=4097), dict(gq=None), dict(gn=None), dict(q=None), dict(q=FAKE + 8), dict(c=None),
               dict(c=FAKE + 2), dict(stride=575), dict(stride=580), dict(out=None), dict(out=FAKE + 4),
               dict(lse=None)):
        assert prefix(L, **kw) == bad, kw
    need = dsa.shared_prefix_workspace_size(par(), kvd(), 1)
    for kw in (dict(ws=None), dict(ws=FAKE + 64), dict(ws_bytes=need - 1)):
        assert prefix(L, **kw) == dsa.DSA_ERR_WORKSPACE, kw


def test_empty_calls_do_nothing(L):
    """Zero tokens or queries: no pointer is needed and nothing is launched
    (there is no GPU here to launch on)."""
    assert rope(L, par_kw=dict(nt=0), x=None, y=None, pos=None) == dsa.DSA_OK
    assert append(L, nt=0, c=None, pe=None, pos=None, slots=None, cache=None) == dsa.DSA_OK
    assert prefix(L, p=par(nq=0), ng=0, gq=None, gn=None, q=None, c=None, out=None, lse=None) == dsa.DSA_OK


@pytest.mark.parametrize("step,call", [("tables", lambda L: tables(L, tab())), ("rope", rope), ("append", append),
                                       ("shared_prefix", prefix)])
def test_host_fault_hook_reaches_the_serving_steps(L, monkeypatch, step, call):
    monkeypatch.setenv("DSA_TEST_INJECT_HOST_ERROR", step)
    assert call(L) == dsa.DSA_ERR_CUDA and "injected host failure in " + step in dsa.last_error()


def test_binding_refuses_what_the_call_would_misread(L):
    """Wrong element types, shapes or devices are refused by the binding."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    ws = torch.zeros(512, dtype=torch.uint8)
    tp = tab(nseq=2, nt=3, max_pages=4, n_free=5)
    ok = dict(seq_len=i32(2), new_len=i32(2), fork_src=None, free_pages=i32(5), free_head=i32(1),
              page_table=i32(2, 4), q_start=i32(3), q_seq=i32(3), positions=i32(3), q_n=i32(3), slots=i32(3),
              kv_len=i32(2), free_head_out=i32(1), ws=ws)
    for name, t in (("seq_len", i32(3)), ("new_len", torch.zeros(2, dtype=torch.int64)), ("page_table", i32(4, 2)),
                    ("slots", i32(2)), ("page_table", i32(4, 2).t()), ("q_start", i32(3))):   # the last: not on a GPU
        with pytest.raises(dsa.DsaError):
            dsa.build_tables(tp, **{**ok, name: t})
    rs, rp = dsa.make_rope_spec(), dsa.make_rope_params(nt=3, h=2, d=64, dtype=dsa.DTYPE_BF16)
    with pytest.raises(dsa.DsaError):
        dsa.rope(rs, rp, torch.zeros(3, 2, 64), i32(3), torch.zeros(3, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(dsa.DsaError):
        dsa.latent_append(rs, torch.zeros(3, 512, dtype=torch.bfloat16), torch.zeros(3, 65, dtype=torch.bfloat16),
                          i32(3), i32(3), torch.zeros(9, 576, dtype=torch.bfloat16), ws)
    with pytest.raises(dsa.DsaError):
        dsa.mla_shared_prefix(par(), kvd(), 1, i32(2), i32(1), torch.zeros(8, 16, 576, dtype=torch.bfloat16), FAKE, 576,
                              FAKE, FAKE, ws)
    with pytest.raises(dsa.DsaError):
        dsa.mla_shared_prefix(par(), kvd(), 2, i32(2), i32(2), FAKE, FAKE, 576, FAKE, FAKE, ws)


@pytest.mark.parametrize("kw", [dict(scaling=dsa.ROPE_SCALE_LINEAR, factor=1e-300),
                                dict(rope_dim=256, theta=1e-300), dict(scaling=dsa.ROPE_SCALE_BASE, factor=1e-300),
                                dict(scaling=dsa.ROPE_SCALE_YARN, factor=1e-306, orig_max_pos=4096)])
def test_speeds_that_are_not_finite_are_refused(L, kw):
    """Their sines would be NaN."""
    assert rope(L, {"rope_dim": 64, **kw}) == dsa.DSA_ERR_INVALID_ARG
    if kw.get("rope_dim", 64) == 64:
        assert append(L, kw) == dsa.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("fp8", [False, True])
def test_strides_of_a_single_row_are_not_looked_at(L, monkeypatch, fp8):
    """One row has no neighbour: whatever stride a tensor of one row reports
    passes the checks (the call then ends at the injected host failure)."""
    monkeypatch.setenv("DSA_TEST_INJECT_HOST_ERROR", "append")
    for cs, ps in ((1, 1), (0, 0), (577, 577), (-3, 5)):
        assert append(L, nt=1, cs=cs, ps=ps, fp8=fp8) == dsa.DSA_ERR_CUDA
        assert append(L, nt=2, cs=cs, ps=ps, fp8=fp8) == dsa.DSA_ERR_INVALID_ARG
