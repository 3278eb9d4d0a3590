"""What the Python binding of the serving operators hands to the C ABI and
what it refuses, argument by argument.  The tensors live on the CPU and say
that they are on GPU 0; the library is a recorder, so nothing is launched."""
import ctypes

import pytest
import torch

from long_context_decode_indexer_b200 import dsa

I32, BF16, FP16, FP32, E4M3 = torch.int32, torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


class On:
    """A CPU tensor that says it is on GPU `dev`."""

    def __init__(self, t, dev=0):
        self.t, self.dev, self.is_cuda = t, dev, True

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


def on(*shape, dtype=I32, dev=0):
    return On(torch.zeros(shape, dtype=dtype), dev)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(dsa, "_lib", r)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return r.calls


def refused(name, fn, *args, **kw):
    """The binding raises for argument `name` and hands nothing on."""
    with pytest.raises(dsa.DsaError, match=name):
        fn(*args, stream=0, **kw)


# ------------------------------------------------------------------ tables
TABLE_ARGS = ("seq_len", "new_len", "fork_src", "free_pages", "free_head", "page_table", "q_start", "q_seq",
              "positions", "q_n", "slots", "kv_len", "free_head_out")


def table_args():
    tp = dsa.make_table_params(nseq=2, nt=3, page_size=64, max_pages=4, n_free=5, cache_rows=6400)
    size = dict(seq_len=2, new_len=2, fork_src=2, free_pages=5, free_head=1, q_start=3, q_seq=3, positions=3, q_n=3,
                slots=3, kv_len=2, free_head_out=1)
    a = {k: on(*((2, 4) if k == "page_table" else (size[k],))) for k in TABLE_ARGS}
    a["ws"] = on(512, dtype=torch.uint8)
    return tp, a


def test_tables_are_handed_on(calls):
    tp, a = table_args()
    dsa.build_tables(tp, **a, stream=0)
    name, args = calls.pop()
    assert name == "dsa_build_tables"
    assert list(args[1:]) == [a[k].data_ptr() for k in TABLE_ARGS] + [a["ws"].data_ptr(), 512, 0]
    dsa.build_tables(tp, **{**a, "fork_src": None}, stream=0)
    assert calls.pop()[1][3] is None


@pytest.mark.parametrize("name", TABLE_ARGS)
def test_table_arguments(calls, name):
    tp, a = table_args()
    shape = tuple(a[name].shape)
    more = shape[:-1] + (shape[-1] + 1,)
    bad = [on(*more), on(*shape, dtype=torch.int64), on(*shape, dtype=FP32), on(*shape, dtype=torch.int16)]
    if shape[-1] > 1:
        bad.append(On(torch.zeros(shape[:-1] + (2 * shape[-1],), dtype=I32)[..., ::2]))
    if name == "page_table":
        bad += [on(4, 2), On(torch.zeros((4, 2), dtype=I32).t())]
    if name != "q_start":          # q_start says which GPU the call is for
        bad += [on(*shape, dev=1), on(*shape, dev=-1)]
    for t in bad:
        refused(name, dsa.build_tables, tp, **{**a, name: t})
    assert not calls


def test_cpu_tensors_and_workspaces_elsewhere(calls):
    tp, a = table_args()
    refused("CUDA device", dsa.build_tables, tp, **{**a, "q_start": on(3, dev=-1)})
    for dev in (-1, 1):
        refused("ws", dsa.build_tables, tp, **{**a, "ws": on(512, dtype=torch.uint8, dev=dev)})
    assert not calls


# -------------------------------------------------------------- other lists
def test_lists_of_the_other_calls(calls):
    rs = dsa.make_rope_spec()
    rp = dsa.make_rope_params(nt=3, h=2, d=64, dtype=dsa.DTYPE_BF16)
    x, y = on(3, 2, 64, dtype=BF16), on(3, 2, 64, dtype=BF16)
    c, pe, cache, ws = on(3, 512, dtype=BF16), on(3, 64, dtype=BF16), on(9, 576, dtype=BF16), on(256, dtype=torch.uint8)
    c8, sc = on(9, 576, dtype=torch.uint8), on(9, dtype=FP32)
    dsa.rope(rs, rp, x, on(3), y, stream=0)
    dsa.latent_append(rs, c, pe, on(3), on(3), cache, ws, stream=0)
    dsa.latent_append_fp8(rs, c, pe, on(3), on(3), c8, sc, ws, stream=0)
    assert [n for n, _ in calls] == ["dsa_rope", "dsa_latent_append", "dsa_latent_append_fp8"]
    calls.clear()
    for bad in (on(4), on(3, dtype=FP32), on(3, dtype=torch.int64)):
        refused("positions", dsa.rope, rs, rp, x, bad, y)
        refused("positions", dsa.rope_backward, rs, rp, x, bad, y)
        refused("positions", dsa.latent_append, rs, c, pe, bad, on(3), cache, ws)
    refused("slots", dsa.latent_append, rs, c, pe, on(3), on(3, dtype=FP32), cache, ws)
    refused("kv_scale", dsa.latent_append_fp8, rs, c, pe, on(3), on(3), c8, on(9), ws)
    refused("kv_scale", dsa.latent_append_fp8, rs, c, pe, on(3), on(3), c8, on(8, dtype=FP32), ws)
    refused("k_pe", dsa.latent_append, rs, c, on(3, 64, dtype=BF16, dev=1), on(3), on(3), cache, ws)
    assert not calls


def prefix_args():
    p = dsa.make_params(nq=8, h_idx=64, d_idx=128, h=16, topk=1, max_n=4096, scale=0.04)
    keep = [torch.zeros(8, dtype=I32), torch.zeros(8, dtype=torch.int64)]
    kv = dsa.make_kv(q_seq=keep[0], q_n=keep[0], seq_row0=keep[1], cache_rows=30)
    a = dict(group_q0=on(3), group_n=on(2), q=on(8, 16, 576, dtype=BF16), kv_cache=on(30, 576, dtype=BF16),
             kv_row_stride=576, out=on(8, 16, 512, dtype=BF16), lse=on(8, 16, dtype=FP32), ws=on(1024, dtype=torch.uint8))
    return p, kv, a, keep


def test_shared_prefix_arguments(calls):
    p, kv, a, keep = prefix_args()
    dsa.mla_shared_prefix(p, kv, 2, **a, stream=0)
    args = calls.pop()[1]
    assert [x for x in args[2:]] == [2] + [a[k].data_ptr() if k != "kv_row_stride" else 576 for k in
                                           ("group_q0", "group_n", "q", "kv_cache", "kv_row_stride", "out", "lse", "ws")] + [1024, 0]
    bad = dict(group_q0=[on(2), on(3, dtype=FP32)], group_n=[on(3), on(2, dtype=FP32), on(2, dev=1)],
               q=[on(8, 16, 576, dtype=FP16), on(16, 8, 576, dtype=BF16), on(8, 16, 512, dtype=BF16),
                  On(torch.zeros((16, 8, 576), dtype=BF16).transpose(0, 1)), on(8, 16, 576, dtype=BF16, dev=-1)],
               out=[on(8, 16, 512, dtype=FP16), on(8, 16, 576, dtype=BF16), on(8, 16, 512, dtype=FP32)],
               lse=[on(8, 16, dtype=BF16), on(16, 8, dtype=FP32), on(8, 16)])
    for name, ts in bad.items():
        for t in ts:
            refused(name, dsa.mla_shared_prefix, p, kv, 2, **{**a, name: t})
    # raw bits of bf16 pass, as everywhere in the binding
    dsa.mla_shared_prefix(p, kv, 2, **{**a, "q": on(8, 16, 576, dtype=torch.int16)}, stream=0)
    assert len(calls) == 1


# -------------------------------------------------------------------- rope
DT = {dsa.DTYPE_BF16: BF16, dsa.DTYPE_FP16: FP16, dsa.DTYPE_FP32: FP32}


def rope_call(rp, x, y, backward):
    if backward:
        dsa.rope_backward(dsa.make_rope_spec(), rp, y, on(rp.nt), x, stream=0)
    else:
        dsa.rope(dsa.make_rope_spec(), rp, x, on(rp.nt), y, stream=0)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
def test_rotated_tensors_that_are_as_described(calls, dtype, backward):
    z = lambda *s: torch.zeros(s, dtype=DT[dtype])
    dense = dsa.make_rope_params(nt=6, h=4, d=64, dtype=dtype)
    wide = z(6, 4, 192)
    views = dsa.make_rope_params(nt=6, h=4, d=64, dtype=dtype, x_strides=(768, 192), y_strides=(768, 192))
    row = z(6, 576)
    shared = dsa.make_rope_params(nt=6, h=4, x_heads=1, d=64, dtype=dtype, x_strides=(576, 64))
    joined = z(6, 300)
    wide_row = dsa.make_rope_params(nt=6, h=4, d=64, dtype=dtype, x_strides=(300, 64))
    one = dsa.make_rope_params(nt=1, h=1, d=64, dtype=dtype, x_strides=(7, 9), y_strides=(0, 0))
    for rp, x, y in ((dense, z(6, 4, 64), z(6, 4, 64)), (dense, z(9, 4, 64), z(6, 256)),
                     (dense, z(2, 3, 4, 64), z(2, 3, 256)), (dense, z(6 * 256), z(7 * 256)),
                     (views, wide[..., 128:], wide[..., 128:]), (shared, row[:, 512:], z(6, 4, 64)),
                     (shared, row[:, None, 512:], z(6, 4, 64)), (wide_row, joined[:, :256], z(6, 4, 64)),
                     (one, z(1, 1, 64), z(1, 64))):
        rope_call(rp, On(x), On(y), backward)
        args = calls.pop()[1]
        assert args[2] == (y if backward else x).data_ptr() and args[4] == (x if backward else y).data_ptr()
    if dtype != dsa.DTYPE_FP32:          # raw bits
        rope_call(dense, On(z(6, 4, 64).view(torch.int16)), On(z(6, 4, 64)), backward)
    rope_call(dsa.make_rope_params(nt=0, h=4, d=64, dtype=dtype), On(z(0, 4, 64)), On(z(0, 4, 64)), backward)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("side", ["x", "y"])
def test_rotated_tensors_that_would_be_misread(calls, side, backward):
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype)
    rp = dsa.make_rope_params(nt=6, h=4, d=64, dtype=dsa.DTYPE_BF16)
    name = ("d" if backward else "") + side
    bad = [On(z(6, 4, 192)[..., 128:]),            # a slice, described as dense
           On(z(4, 6, 64)), On(z(4, 6, 64).transpose(0, 1)), On(z(6, 64, 4).transpose(1, 2)),
           On(z(5, 4, 64)), On(z(6, 4, 63)), On(z(6, 3, 64)), On(z(6, 128)), On(z(6 * 256 - 1)),
           On(z(6, 4, 128)[..., ::2]), On(z(1, 4, 64).expand(6, 4, 64)), On(z(6, 8, 64)[:, ::2]),
           On(z(2, 3, 4, 128)[..., :64]), On(z(3, 4, 64)), On(z(24, 64)),
           On(z(6, 4, 64, dtype=FP16)), On(z(6, 4, 64, dtype=FP32)), On(z(6, 4, 64, dtype=torch.int32)),
           On(z(6, 4, 64), dev=1), On(z(6, 4, 64), dev=-1)]
    ok = On(z(6, 4, 64))
    for t in bad:
        with pytest.raises(dsa.DsaError, match="^" + name + ":"):
            rope_call(rp, t if side == "x" else ok, t if side == "y" else ok, backward)
    # a short buffer for strides that reach past it
    far = dsa.make_rope_params(nt=6, h=4, d=64, dtype=dsa.DTYPE_BF16, x_strides=(512, 64), y_strides=(512, 64))
    with pytest.raises(dsa.DsaError, match="^" + name + ":"):
        rope_call(far, On(z(6 * 256) if side == "x" else z(6 * 512)), On(z(6 * 256) if side == "y" else z(6 * 512)), backward)
    assert not calls
    with pytest.raises(dsa.DsaError, match="dtype"):
        rope_call(dsa.make_rope_params(nt=6, h=4, d=64, dtype=3), ok, ok, backward)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("fp8", [False, True])
def test_append_caches(calls, fp8):
    dt = torch.uint8 if fp8 else BF16
    ws, sc = on(256, dtype=torch.uint8), on(64, dtype=FP32)
    kv_a = torch.zeros((3, 576), dtype=BF16)
    name = "kv8_cache" if fp8 else "kv_cache"

    def append(cache, c=On(kv_a[:, :512]), pe=On(kv_a[:, 512:])):
        if fp8:
            dsa.latent_append_fp8(dsa.make_rope_spec(), c, pe, on(3), on(3), cache, sc, ws, stream=0)
        else:
            dsa.latent_append(dsa.make_rope_spec(), c, pe, on(3), on(3), cache, ws, stream=0)

    z = lambda *s, dtype=dt: torch.zeros(s, dtype=dtype)
    good = [z(64, 576), z(64, 640), z(64, 640)[:, :576], z(64, 704)[:, 64:]]
    good += [z(64, 576, dtype=E4M3)] if fp8 else [z(64, 576, dtype=torch.int16)]
    for t in good:
        append(On(t))
        args = calls.pop()[1]
        assert args[8:10] == (t.data_ptr(), t.stride(0)) and args[-4] == 64
        assert args[2:6] == (kv_a.data_ptr(), 576, kv_a.data_ptr() + 1024, 576)
    bad = [z(4, 16, 576),                       # pages: rows of one would be 16 apart
           z(64, 512), z(640, 64).t(), z(64, 1152)[:, ::2], z(64 * 576), z(64, 640)[:, 128:],
           z(64, 576, dtype=FP16), z(64, 576, dtype=FP32), z(64, 576, dtype=BF16 if fp8 else torch.uint8)]
    for t in [On(t) for t in bad] + [on(64, 576, dtype=dt, dev=1), on(64, 576, dtype=dt, dev=-1)]:
        with pytest.raises(dsa.DsaError, match="^%s:" % name):
            append(t)
    for part, w in (("c_kv", 512), ("k_pe", 64)):
        for t in (z(3, w, dtype=FP16), z(3, w + 8, dtype=BF16), z(4, w, dtype=BF16), z(w, 3, dtype=BF16).t(),
                  z(3, w, 1, dtype=BF16)):
            with pytest.raises(dsa.DsaError, match="^%s:" % part):
                append(On(good[0]), **{"c" if part == "c_kv" else "pe": On(t)})
    assert not calls


# ----------------------------------------------------------- shared prefix
def test_shared_prefix_caches(calls):
    p, kv, a, keep = prefix_args()          # 30 rows
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype)
    for t, stride in ((z(30, 576), 576), (z(31, 640), 640), (z(30, 640)[:, :576], 640), (z(2, 15, 576), 576),
                      (z(29 * 584 + 576), 584), (z(30, 576, dtype=torch.int16), 576)):
        dsa.mla_shared_prefix(p, kv, 2, **{**a, "kv_cache": On(t), "kv_row_stride": stride}, stream=0)
        assert calls.pop()[1][6:8] == (t.data_ptr(), stride)
    bad = [(on(30, 576, dtype=torch.uint8), 576),       # an FP8 cache: rows half as long
           (on(30, 576, dtype=E4M3), 576), (on(30, 576, dtype=FP16), 576), (on(30, 576, dtype=FP32), 576),
           (on(30, 576, dtype=BF16, dev=-1), 576), (on(30, 576, dtype=BF16, dev=1), 576),
           (on(29, 576, dtype=BF16), 576), (on(30, 640, dtype=BF16), 576), (on(30, 576, dtype=BF16), 640),
           (on(30, 512, dtype=BF16), 512), (on(29 * 576 + 575, dtype=BF16), 576), (on(30, 1, 576, dtype=BF16), 640),
           (On(z(2, 20, 576)[:, :15]), 576), (On(z(576, 30).t()), 576), (On(z(30, 1152)[:, ::2]), 1152)]
    for t, stride in bad:
        refused("kv_cache", dsa.mla_shared_prefix, p, kv, 2, **{**a, "kv_cache": t, "kv_row_stride": stride})
    assert not calls
    dsa.mla_shared_prefix(p, kv, 2, **{**a, "kv_cache": 1 << 20}, stream=0)     # an address, as it is
    assert calls.pop()[1][6] == 1 << 20


def test_shared_prefix_of_no_queries_needs_no_tensors(calls):
    p, kv, a, keep = prefix_args()
    p = dsa.make_params(nq=0, h_idx=64, d_idx=128, h=16, topk=1, max_n=4096, scale=0.04)
    dsa.mla_shared_prefix(p, kv, 0, on(1), None, None, None, 576, None, None, a["ws"], stream=0)
    assert calls.pop()[1][5:8] == (None, None, 576)


def test_views_of_several_token_or_page_dimensions(calls):
    """[batch, length, heads, width] and its slices, [pages, size, 1, width]:
    evenly spaced rows are what they are, whatever they are called."""
    z = lambda *s: torch.zeros(s, dtype=BF16)
    wide = z(2, 3, 4, 192)
    rp = dsa.make_rope_params(nt=6, h=4, d=64, dtype=dsa.DTYPE_BF16, x_strides=(768, 192), y_strides=(768, 192))
    k = z(2, 3, 1, 576)
    shared = dsa.make_rope_params(nt=6, h=4, x_heads=1, d=64, dtype=dsa.DTYPE_BF16, x_strides=(576, 576))
    flat = z(2, 3, 300)
    joined = dsa.make_rope_params(nt=6, h=4, d=64, dtype=dsa.DTYPE_BF16, x_strides=(300, 64))
    for r, x, y in ((rp, wide[..., 128:], wide[..., :64]), (rp, z(6, 1, 4, 192)[..., 64:128], z(1, 6, 4, 192)[..., :64]),
                    (shared, k[..., 512:], z(2, 3, 4, 64)), (shared, k[..., 0, 512:], z(2, 3, 256)),
                    (joined, flat[..., :256], z(6, 4, 64))):
        rope_call(r, On(x), On(y), False)
        assert calls.pop()[1][2] == x.data_ptr()
    for x in (wide[:, :2, :, 128:], wide.transpose(0, 1)[..., 128:], wide[..., 128:].transpose(1, 2), wide[:, ::2, :, :64]):
        with pytest.raises(dsa.DsaError, match="^x:"):
            rope_call(rp, On(x), On(wide[..., :64]), False)
    for x in (z(6, 7, 64), z(2, 3, 7, 64), z(1, 7, 64), z(12, 1, 64)[::2]):     # one head is asked for
        r = dsa.make_rope_params(nt=x.shape[0], h=4, x_heads=1, d=64, dtype=dsa.DTYPE_BF16)
        with pytest.raises(dsa.DsaError, match="^x:"):
            rope_call(r, On(x), On(z(x.shape[0], 4, 64)), False)
    p, kv, a, keep = prefix_args()
    for t in (z(2, 16, 1, 576), z(1, 30, 576), z(30, 1, 1, 576), z(3, 10, 600)[..., :576]):
        stride = t.stride(-3) if t.shape[-2] == 1 else t.stride(-2)
        dsa.mla_shared_prefix(p, kv, 2, **{**a, "kv_cache": On(t), "kv_row_stride": stride}, stream=0)
        assert calls.pop()[1][6:8] == (t.data_ptr(), stride)
    refused("kv_cache", dsa.mla_shared_prefix, p, kv, 2, **{**a, "kv_cache": On(z(2, 16, 2, 576)[:, :, 0]), "kv_row_stride": 576})
    assert not calls
