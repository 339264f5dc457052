"""moe_serve.h: the library exports what it declares, the binding knows every symbol, and bad arguments are
refused before anything is launched (no GPU needed: these calls return before touching CUDA)."""
import ctypes
import os
import re

import pytest

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "moe_serve.h")
A = 1 << 20  # a fake, never-dereferenced address


@pytest.fixture(scope="module")
def moe():
    import mxfp4_routed_expert_moe_gb300 as m
    import mxfp4_routed_expert_moe_gb300.build as b
    b.build()
    m.lib()
    return m


@pytest.fixture(scope="module")
def serve(moe):
    from mxfp4_routed_expert_moe_gb300 import serve as s
    s._lib()
    return s


def test_header_binding_and_library_agree(moe):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(moe_\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(moe.SERVE_EXPORTS)
    L = ctypes.CDLL(moe.LIB_PATH)
    for name in names:
        assert hasattr(L, name), name
    assert moe.SAMPLE_MAX_VOCAB == int(re.search(r"MOE_SAMPLE_MAX_VOCAB (\d+)", src).group(1))
    assert moe.SERVE_MAX_BATCH == int(re.search(r"MOE_SERVE_MAX_BATCH (\d+)", src).group(1))


def cache(serve, **kw):
    c = serve._Cache(A, A, 10, 16, 2, 64, 16 * 2 * 64, 2 * 64, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(serve, **kw):
    b = serve._Batch(3, 3, 1, 4, 4, 0, None, A, A, None)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


BAD_CACHE = [(dict(k=None), 1), (dict(v=A + 8), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1),
             (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(head_dim=96), 2), (dict(kv_heads=0), 1),
             (dict(kv_heads=257), 2), (dict(token_stride=132), 1), (dict(page_stride=-8), 1), (dict(head_stride=1 << 40), 2)]
BAD_BATCH = [(dict(batch=0), 1), (dict(batch=4097, tokens=4097), 2), (dict(tokens=0), 1), (dict(tokens=4), 1), (dict(max_q=0), 1),
             (dict(kv_len=None), 1), (dict(table=A + 2), 1), (dict(table_stride=3), 1), (dict(prefix_len=5), 1),
             (dict(prefix_len=-1, prefix_table=A), 1), (dict(q_start=A + 1), 1)]


def append(serve, c, b, dtype=1, q=A, k=A, v=A, q_heads=4, qs=256, ks=128, vs=128, q_out=A, os=256, rope=A, rows=9,
           rot=64, inter=0, status=None):
    return serve._lib().moe_kv_append(ctypes.byref(c), ctypes.byref(b), dtype, q, k, v, q_heads, qs, ks, vs, q_out, os,
                                      rope, rows, rot, inter, status, None)


def attend(serve, c, b, q=A, q_heads=4, qs=256, scale=1.0, out=A, os=256, lse=None, ws=A, n=1 << 40, status=None):
    return serve._lib().moe_prefix_attention(ctypes.byref(c), ctypes.byref(b), q, q_heads, qs, scale, out, os, lse, ws,
                                             n, status, None)


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_bad_cache_is_refused(serve, kw, want):
    c, b = cache(serve, **kw), batch(serve)
    assert append(serve, c, b) == want
    assert attend(serve, c, b) == want
    assert serve._lib().moe_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 4) == 0


@pytest.mark.parametrize("kw,want", BAD_BATCH)
def test_bad_batch_is_refused(serve, kw, want):
    c, b = cache(serve), batch(serve, **kw)
    assert append(serve, c, b) == want
    assert attend(serve, c, b) == want
    assert serve._lib().moe_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 4) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), 1), (dict(k=None), 1), (dict(v=A + 4), 1), (dict(ks=132), 1), (dict(dtype=0, vs=130), 1),
    (dict(q_out=None), 1), (dict(q=None), 1), (dict(q_heads=3), 1), (dict(q_heads=2048), 2), (dict(os=252), 1),
    (dict(rot=8), 1), (dict(rot=80), 1), (dict(rot=-16), 1), (dict(rope=None), 1), (dict(rope=A + 4), 1),
    (dict(rows=0), 1), (dict(inter=2), 1), (dict(status=A + 2), 1)])
def test_append_refusals(serve, kw, want):
    assert append(serve, cache(serve), batch(serve), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(q=A + 8), 1), (dict(out=A + 2), 1), (dict(qs=260), 1), (dict(os=4), 1),
    (dict(q_heads=5), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(lse=A + 1), 1), (dict(ws=None), 1), (dict(ws=A + 16), 1), (dict(n=1000), 3),
    (dict(status=A + 3), 1)])
def test_attention_refusals(serve, kw, want):
    assert attend(serve, cache(serve), batch(serve), **kw) == want


def test_null_structs_are_refused(serve):
    L = serve._lib()
    assert L.moe_kv_append(None, ctypes.byref(batch(serve)), 1, A, A, A, 4, 256, 128, 128, A, 256, A, 9, 64, 0, None, None) == 1
    assert L.moe_prefix_attention(ctypes.byref(cache(serve)), None, A, 4, 256, 1.0, A, 256, None, A, 1 << 40, None, None) == 1


def test_workspace_grows_with_the_batch(serve):
    L = serve._lib()
    size = lambda **kw: L.moe_attention_workspace_bytes(ctypes.byref(cache(serve)), ctypes.byref(batch(serve, **kw)), 8)  # noqa: E731
    small, big = size(), size(batch=300, tokens=300)
    assert 0 < small < big and small % 256 == 0
    assert size(q_start=A, tokens=900, max_q=300) > 0
    assert size(prefix_len=100, prefix_table=A) >= small


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 1), (dict(vocab=0), 1), (dict(vocab=(1 << 18) + 1, stride=1 << 20), 2), (dict(logits=None), 1),
    (dict(logits=A + 2), 1), (dict(dtype=0, logits=A + 2), 1), (dict(dtype=1, logits=A + 1), 1), (dict(dtype=7), 1),
    (dict(stride=99), 1), (dict(u=None), 1), (dict(token=None), 1), (dict(token=A + 2), 1), (dict(top_k=A + 1), 1),
    (dict(probs=A + 2), 1)])
def test_sample_refusals(serve, kw, want):
    a = dict(rows=2, vocab=100, logits=A, dtype=0, stride=100, u=A, temperature=None, top_k=None, top_p=None, min_p=None,
             token=A, logprob=None, kept=None, probs=None) | kw
    assert serve._lib().moe_sample(*a.values(), None) == want


def test_binding_checks_shapes_and_types(moe):
    import torch as t
    k = t.zeros(10, 16, 2, 64, dtype=t.bfloat16)
    with pytest.raises(TypeError):
        moe.KVCache(k.float(), k.float())
    with pytest.raises(ValueError):
        moe.KVCache(k, k[:9])
    with pytest.raises(ValueError):
        moe.KVCache(k.transpose(2, 3), k.transpose(2, 3))
    c = moe.KVCache(k.transpose(1, 2).contiguous().transpose(1, 2), k.transpose(1, 2).contiguous().transpose(1, 2))
    assert (c.struct.page_size, c.struct.token_stride, c.struct.head_stride) == (16, 64, 16 * 64)
    i32 = lambda *x: t.zeros(*x, dtype=t.int32)  # noqa: E731
    with pytest.raises(ValueError):
        moe.KVBatch(i32(3), i32(2, 4))
    with pytest.raises(TypeError):
        moe.KVBatch(i32(3).long(), i32(3, 4))
    with pytest.raises(TypeError):
        moe.KVBatch(i32(3), i32(3, 4).long())
    with pytest.raises(ValueError):
        moe.KVBatch(i32(3), i32(3, 4), q_start=i32(3))
    with pytest.raises(ValueError):
        moe.KVBatch(i32(3), i32(3, 4), prefix_len=5)
    b = moe.KVBatch(i32(3), i32(3, 4), prefix_table=i32(2), prefix_len=33)
    q = t.zeros(3, 4, 64, dtype=t.bfloat16)
    ws = t.zeros(256, dtype=t.uint8)
    with pytest.raises(ValueError):  # 33 tokens in two pages of 16
        moe.prefix_attention(c, b, q, q, ws, stream=0)
    b = moe.KVBatch(i32(3), i32(3, 4))
    with pytest.raises(TypeError):
        moe.prefix_attention(c, b, q.float(), q, ws, stream=0)
    with pytest.raises(ValueError):
        moe.prefix_attention(c, b, q.transpose(1, 2), q, ws, stream=0)
    with pytest.raises(ValueError):
        moe.prefix_attention(c, b, q[:2], q[:2], ws, stream=0)
    with pytest.raises(moe.MoeError):
        moe.attention_workspace_bytes(c, b, 3)
    kv = t.zeros(3, 2, 64, dtype=t.bfloat16)
    with pytest.raises(TypeError):
        moe.kv_append(c, b, kv, kv.float(), stream=0)
    with pytest.raises(ValueError):
        moe.kv_append(c, b, kv[:, :1], kv, stream=0)
    with pytest.raises(ValueError):
        moe.kv_append(c, b, kv, kv, rope=t.zeros(5, 32), rot_dim=64, stream=0)
    x, u, tok = t.zeros(3, 50), t.zeros(3), i32(3)
    with pytest.raises(TypeError):
        moe.sample(x.half(), u, tok, stream=0)
    with pytest.raises(ValueError):
        moe.sample(x, u[:2], tok, stream=0)
    with pytest.raises(TypeError):
        moe.sample(x, u, tok.long(), stream=0)
    with pytest.raises(TypeError):
        moe.sample(x, u, tok, top_k=u, stream=0)
    with pytest.raises(ValueError):
        moe.sample(x.t(), u, tok, stream=0)


def test_lengths_past_what_attention_counts_are_refused(serve, moe):
    assert re.search(r"MOE_SERVE_MAX_LEN \(1 << 30\)", open(HEADER).read()) and moe.SERVE_MAX_LEN == 1 << 30
    c, b = cache(serve), batch(serve, prefix_len=moe.SERVE_MAX_LEN + 1, prefix_table=A)
    assert append(serve, c, b) == 2 and attend(serve, c, b) == 2
    assert serve._lib().moe_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 4) == 0


@pytest.mark.parametrize("kw", [
    dict(batch=1, tokens=2, q_start=A, prefix_len=32768, prefix_table=A), dict(batch=2, tokens=2, q_start=A, prefix_len=200, prefix_table=A),
    dict(batch=1, tokens=1, prefix_len=100, prefix_table=A), dict(batch=1, tokens=1), dict(batch=3, tokens=3)])
@pytest.mark.parametrize("group", [1, 7])
def test_max_q_past_what_the_batch_can_have_changes_no_plan(serve, kw, group):
    """max_q is an upper bound: no sequence has more new tokens than the batch, nor more than one without q_start.
    Own parts planned by a larger bound went to the other side of the split kernel than the prefix."""
    L = serve._lib()
    most = kw["tokens"] if "q_start" in kw else 1
    size = lambda m: L.moe_attention_workspace_bytes(ctypes.byref(cache(serve)), ctypes.byref(batch(serve, max_q=m, **kw)), 2 * group)  # noqa: E731
    assert 0 < size(most) == size(8) == size(100) == size((1 << 31) - 1)


def test_tensors_off_the_gpu_are_refused(moe, monkeypatch):
    """Each tensor argument of a call has to be on the cache's (or the logits') GPU: a host address is not followed.
    Nothing is launched here, whatever the checks say."""
    import torch as t
    from mxfp4_routed_expert_moe_gb300 import serve as s

    class Gpu(t.Tensor):  # a host tensor that says it is on device 0
        def get_device(self):
            return 0

    calls = []
    fake = type("L", (), {n: staticmethod(lambda *a, n=n: calls.append(n) or 0) for n in moe.SERVE_EXPORTS})()
    s._lib()
    monkeypatch.setattr(s, "_READY", fake)
    gpu = lambda x: x.as_subclass(Gpu)  # noqa: E731
    bf = lambda *x: t.zeros(*x, dtype=t.bfloat16)  # noqa: E731
    i32 = lambda *x: t.zeros(*x, dtype=t.int32)  # noqa: E731

    def refused(f, args, launch):
        """Fails with every single argument on the host, passes with none."""
        f(**{k: gpu(v) for k, v in args.items()})
        assert calls == [launch]
        calls.clear()
        for name in args:
            with pytest.raises(ValueError):
                f(**{k: v if k == name else gpu(v) for k, v in args.items()})
            assert not calls, name

    def batch_of(kv_len, table, q_start, prefix_table):
        return moe.KVBatch(kv_len, table, tokens=3, q_start=q_start, prefix_table=prefix_table, prefix_len=20)

    here = dict(ck=bf(10, 16, 2, 64), cv=bf(10, 16, 2, 64), kv_len=i32(3), table=i32(3, 4), q_start=i32(4), prefix_table=i32(2))

    def append(ck, cv, kv_len, table, q_start, prefix_table, **kw):
        moe.kv_append(moe.KVCache(ck, cv), batch_of(kv_len, table, q_start, prefix_table), rot_dim=64, stream=0, **kw)

    refused(append, here | dict(k=bf(3, 2, 64), v=bf(3, 2, 64), q=bf(3, 4, 64), q_out=bf(3, 4, 64), rope=t.zeros(9, 64),
                                status=i32(1)), "moe_kv_append")

    def attend(ck, cv, kv_len, table, q_start, prefix_table, **kw):
        moe.prefix_attention(moe.KVCache(ck, cv), batch_of(kv_len, table, q_start, prefix_table), stream=0, **kw)

    refused(attend, here | dict(q=bf(3, 4, 64), out=bf(3, 4, 64), ws=t.zeros(256, dtype=t.uint8), lse=t.zeros(3, 4),
                                status=i32(1)), "moe_prefix_attention")
    refused(lambda **kw: moe.sample(stream=0, **kw),
            dict(logits=t.zeros(3, 50), u=t.zeros(3), token=i32(3), temperature=t.zeros(3), top_k=i32(3), top_p=t.zeros(3),
                 min_p=t.zeros(3), logprob=t.zeros(3), kept=i32(3), probs=t.zeros(3, 50)), "moe_sample")


def test_workspace_and_status_of_another_form_are_refused(serve, moe):
    import torch as t
    c = moe.KVCache(t.zeros(10, 16, 2, 64, dtype=t.bfloat16), t.zeros(10, 16, 2, 64, dtype=t.bfloat16))
    b = moe.KVBatch(t.zeros(3, dtype=t.int32), t.zeros(3, 4, dtype=t.int32))
    q = t.zeros(3, 4, 64, dtype=t.bfloat16)
    with pytest.raises(ValueError, match="ws"):  # one byte, said to be many
        moe.prefix_attention(c, b, q, q, t.zeros(1, dtype=t.uint8).expand(1 << 30), stream=0)
    with pytest.raises(TypeError, match="status"):
        moe.prefix_attention(c, b, q, q, t.zeros(256, dtype=t.uint8), status=t.zeros(1, dtype=t.int64), stream=0)


@pytest.mark.parametrize("kw", [dict(os=0), dict(os=248), dict(os=-248), dict(q_out=A, q=A, qs=512, os=256),
                                dict(q_out=A, q=A, dtype=0, qs=256, os=256)])
def test_append_refuses_query_rows_over_one_another(serve, kw):
    """Rows of q_out that overlap, or that lie over rows of q other than their own, would hold what came last."""
    assert append(serve, cache(serve), batch(serve), **kw) == 1


@pytest.mark.parametrize("os", [0, 248, -248])
def test_attention_refuses_result_rows_over_one_another(serve, os):
    assert attend(serve, cache(serve), batch(serve), os=os) == 1


def test_a_scale_past_the_range_of_its_base_2_form_is_refused(serve):
    """The kernels take scale log2(e): of a finite scale above 2.36e38 it is infinite, and 0 times it NaN."""
    assert attend(serve, cache(serve), batch(serve), scale=3e38) == 1
