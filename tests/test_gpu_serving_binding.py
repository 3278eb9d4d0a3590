"""The binding's refusals on GPU tensors: the call as it should be goes
through, the same call with one argument that would be misread is refused
before anything is launched (the outputs stay as they were)."""
import pytest
import torch

from conftest import cuda_ok
from long_context_decode_indexer_b200 import dsa
from long_context_decode_indexer_b200.batch import workspace

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

BF16 = torch.bfloat16


def z(*s, dtype=torch.int32, device="cuda"):
    return torch.zeros(s, dtype=dtype, device=device)


def one_at_a_time(fn, ok, bad, outputs):
    """fn(**ok) runs; with each of `bad` (name, value) it raises for that name."""
    fn(**ok)
    torch.cuda.synchronize()
    before = {k: ok[k].clone() for k in outputs}
    for name, value in bad:
        with pytest.raises(dsa.DsaError, match="^%s:" % name):
            fn(**{**ok, name: value})
    torch.cuda.synchronize()
    for k, v in before.items():
        assert torch.equal(ok[k], v), k


def test_tables():
    tp = dsa.make_table_params(nseq=2, nt=3, page_size=64, max_pages=4, n_free=5, cache_rows=6400)
    ok = dict(seq_len=z(2), new_len=z(2) + 1, fork_src=None, free_pages=torch.arange(5, dtype=torch.int32, device="cuda"),
              free_head=z(1), page_table=z(2, 4), q_start=z(3), q_seq=z(3), positions=z(3), q_n=z(3), slots=z(3),
              kv_len=z(2), free_head_out=z(1), ws=workspace(512))
    one_at_a_time(lambda **a: dsa.build_tables(tp, **a), ok,
                  [("seq_len", z(3)), ("seq_len", z(2, dtype=torch.int64)), ("new_len", z(2, dtype=torch.float32)),
                   ("page_table", z(4, 2)), ("page_table", z(4, 2).t()), ("slots", z(6)[::2]), ("q_n", z(3, device="cpu"))],
                  ("page_table", "slots", "kv_len"))
    assert ok["slots"].tolist() == [0, 64, -1]


@pytest.mark.parametrize("backward", [False, True])
def test_rope(backward):
    rs, rp = dsa.make_rope_spec(), dsa.make_rope_params(nt=6, h=4, d=64, dtype=dsa.DTYPE_BF16)
    src, dst = ("dy", "dx") if backward else ("x", "y")
    q = torch.randn(6, 4, 192, device="cuda").to(BF16)
    ok = {src: torch.randn(6, 4, 64, device="cuda").to(BF16), dst: z(6, 4, 64, dtype=BF16), "positions": z(6) + 5}
    bad = [(k, t) for k in (src, dst) for t in (q[..., 128:], z(4, 6, 64, dtype=BF16).transpose(0, 1), z(5, 4, 64, dtype=BF16),
                                                z(6, 4, 64, dtype=torch.float16), z(6, 4, 64, dtype=BF16, device="cpu"))]
    fn = dsa.rope_backward if backward else dsa.rope
    one_at_a_time(lambda **a: fn(rs, rp, a[src], a["positions"], a[dst]), ok,
                  bad + [("positions", z(6, dtype=torch.float32)), ("positions", z(7))], (src, dst))
    # the slice as what it is
    rp = dsa.make_rope_params(nt=6, h=4, d=64, dtype=dsa.DTYPE_BF16, x_strides=(768, 192), y_strides=(768, 192))
    keep = q.clone()
    fn(rs, rp, q[..., 128:], z(6) + 5, q[..., 128:])
    assert torch.equal(q[..., :128], keep[..., :128]) and not torch.equal(q, keep)


@pytest.mark.parametrize("fp8", [False, True])
def test_append(fp8):
    rs, kv_a, ws = dsa.make_rope_spec(), torch.randn(3, 576, device="cuda").to(BF16), workspace(dsa.WS_STATUS_BYTES)
    dt, name = (torch.uint8, "kv8_cache") if fp8 else (BF16, "kv_cache")
    ok = {"c_kv": kv_a[:, :512], "k_pe": kv_a[:, 512:], "positions": z(3), "slots": torch.tensor([63, 0, 7], dtype=torch.int32, device="cuda"),
          name: z(64, 576, dtype=dt)}
    bad = [(name, t) for t in (z(4, 16, 576, dtype=dt), z(64, 640, dtype=dt)[:, 128:], z(64, 1152, dtype=dt)[:, ::2],
                               z(64, 576, dtype=torch.float16), z(64, 576, dtype=dt, device="cpu"))]
    bad += [("k_pe", kv_a[:, 500:564].half()), ("slots", z(3, dtype=torch.float32))]
    if fp8:
        ok["kv_scale"] = z(64, dtype=torch.float32)
        bad += [("kv_scale", z(63, dtype=torch.float32)), ("kv_scale", z(64))]
        fn = dsa.latent_append_fp8
    else:
        fn = dsa.latent_append
    one_at_a_time(lambda **a: fn(rs, ws=ws, **a), ok, bad, (name,))
    assert dsa.check_status(ws) == dsa.DSA_OK
    touched = ok[name].float().abs().sum(1) != 0 if not fp8 else ok[name].any(1)
    assert sorted(torch.nonzero(touched)[:, 0].tolist()) == [0, 7, 63]


def test_shared_prefix():
    p = dsa.make_params(nq=2, h_idx=64, d_idx=128, h=4, topk=1, max_n=128, scale=0.04)
    q_seq, q_n, table = z(2), z(2) + 100, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    kv = dsa.make_kv(q_seq=q_seq, q_n=q_n, page_table=table, page_size=64, cache_rows=128)
    cache = torch.randn(128, 576, device="cuda").to(BF16)
    ok = dict(group_q0=torch.tensor([0, 2], dtype=torch.int32, device="cuda"), group_n=z(1) + 70,
              q=torch.randn(2, 4, 576, device="cuda").to(BF16), kv_cache=cache, out=z(2, 4, 512, dtype=BF16),
              lse=z(2, 4, dtype=torch.float32), ws=workspace(dsa.shared_prefix_workspace_size(p, kv, 1)))
    call = lambda **a: dsa.mla_shared_prefix(p, kv, 1, **a, kv_row_stride=576)
    one_at_a_time(call, ok, [("kv_cache", cache.cpu()), ("kv_cache", z(128, 576, dtype=torch.uint8)), ("kv_cache", cache[:127]),
                             ("kv_cache", cache.half()), ("kv_cache", z(128, 640, dtype=BF16)), ("q", ok["q"].half()),
                             ("out", z(2, 4, 512, dtype=torch.float32)), ("lse", z(2, 4)), ("group_n", z(1, dtype=torch.float32))],
                  ("out", "lse"))
    assert dsa.check_status(ok["ws"]) == dsa.DSA_OK
    flat = ok["out"].clone()
    call(**{**ok, "kv_cache": cache.view(2, 64, 576)})       # pages, as they lie
    assert torch.equal(ok["out"], flat)
