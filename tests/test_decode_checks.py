"""What the paged-cache calls refuse (no GPU: moss_enc_paged_refusal is pure),
and what the Python binding refuses before it calls the library."""
import ctypes
import types

import pytest

from audio_encoder_b200 import binding

torch = pytest.importorskip("torch")

P = 1 << 20  # an aligned address that nothing dereferences


def cache(**kw):
    d = dict(k=P, v=P, page_table=P, table_stride=4, stride_page=16 * 8 * 128, stride_token=8 * 128, stride_head=128,
             n_seqs=3, pages_per_seq=4, n_pages=12, page_size=16, n_kv_heads=8, head_dim=128, dtype=binding.KV_BF16,
             k_scale=1.0, v_scale=1.0)
    return binding.KVCacheDesc(**{**d, **kw})


def rows(**kw):
    d = dict(k=P, v=P, q=P, q_out=P, k_stride=1024, v_stride=1024, q_stride=2048, q_out_stride=2048, positions=P, seqs=P,
             inv_freq=P, n_rows=5, n_q_heads=16, dtype=binding.KV_BF16, rotary=128, interleaved=0)
    return binding.KVRows(**{**d, **kw})


def attn(**kw):
    d = dict(q=P, out=P, lse=P, lengths=P, q_stride=2048, n_q_heads=16, dtype=binding.KV_BF16, scale=0.1, max_len=0,
             workspace=None, workspace_bytes=0)
    return binding.Attn(**{**d, **kw})


def refusal(c=None, r=None, a=None):
    ref = [None if x is None else ctypes.byref(x) for x in (c, r, a)]
    why = binding.lib().moss_enc_paged_refusal(*ref)
    return None if why is None else why.decode()


def test_plain_arguments_are_taken():
    assert refusal(cache()) is None
    assert refusal(cache(), rows()) is None
    assert refusal(cache(), None, attn()) is None
    assert refusal(None) == "no cache"


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(head_dim=96), dict(head_dim=0), dict(n_seqs=-1), dict(n_kv_heads=0),
    dict(n_pages=0), dict(pages_per_seq=0), dict(page_size=8), dict(page_size=48), dict(page_size=0),
    dict(page_size=1 << 20, pages_per_seq=(1 << 10) + 1, table_stride=1 << 11), dict(k=None), dict(v=None), dict(page_table=None), dict(k=P + 8),
    dict(v=P + 2), dict(page_table=P + 2), dict(stride_token=1028), dict(stride_token=64), dict(stride_head=64),
    dict(stride_head=132), dict(stride_page=-2048), dict(stride_page=4), dict(stride_page=1 << 59), dict(stride_token=1 << 58), dict(table_stride=3),
    dict(dtype=binding.KV_E4M3, k_scale=0.0), dict(dtype=binding.KV_E4M3, v_scale=-1.0),
    dict(dtype=binding.KV_E4M3, k_scale=float("nan")), dict(dtype=binding.KV_E4M3, v_scale=float("inf")),
    dict(dtype=binding.KV_E4M3, k_scale=1e-45), dict(dtype=binding.KV_E4M3, stride_head=136)])
def test_caches_that_are_refused(kw):
    assert refusal(cache(**kw))


@pytest.mark.parametrize("kw", [
    dict(n_seqs=0, page_table=None), dict(n_pages=1, stride_page=0), dict(stride_page=1 << 40), dict(n_kv_heads=1, stride_head=0),
    dict(n_seqs=1, table_stride=0), dict(k_scale=0.0), dict(dtype=binding.KV_E4M3, k_scale=0.5),
    dict(stride_token=128, stride_head=16 * 128), dict(page_size=1 << 20, pages_per_seq=1 << 10, table_stride=1 << 11)])
def test_caches_that_are_taken(kw):
    assert refusal(cache(**kw)) is None


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(n_rows=(1 << 30) + 1), dict(n_q_heads=-1), dict(dtype=binding.KV_F16), dict(dtype=binding.KV_E4M3), dict(rotary=8),
    dict(rotary=144), dict(rotary=-16), dict(inv_freq=None), dict(inv_freq=P + 4), dict(interleaved=2),
    dict(k_stride=1028), dict(k_stride=512), dict(q_stride=1024), dict(q_out_stride=2052), dict(k=None), dict(v=None),
    dict(positions=None), dict(q=None), dict(q_out=None), dict(k=P + 8), dict(q_out=P + 4), dict(positions=P + 1),
    dict(seqs=P + 2), dict(q_out_stride=4096), dict(seqs=None)])
def test_rows_that_are_refused(kw):
    assert refusal(cache(), rows(**kw))


@pytest.mark.parametrize("kw", [
    dict(n_rows=0, k=None, v=None, q=None, q_out=None, positions=None), dict(n_q_heads=0, q=None, q_out=None),
    dict(rotary=0, inv_freq=None), dict(rotary=16, interleaved=1), dict(n_rows=1, k_stride=0), dict(n_rows=3, seqs=None)])
def test_rows_that_are_taken(kw):
    assert refusal(cache(), rows(**kw)) is None


def test_rows_of_either_type_meet_an_e4m3_cache():
    c = cache(dtype=binding.KV_E4M3)
    assert refusal(c, rows()) is None and refusal(c, rows(dtype=binding.KV_F16)) is None
    assert refusal(c, None, attn(dtype=binding.KV_F16)) is None
    assert refusal(c, rows(dtype=binding.KV_E4M3)) and refusal(c, None, attn(dtype=binding.KV_E4M3))


@pytest.mark.parametrize("kw", [
    dict(n_q_heads=0), dict(n_q_heads=12), dict(max_len=-1), dict(dtype=binding.KV_F16), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(q_stride=1024), dict(q_stride=2052), dict(q=None), dict(out=None), dict(lengths=None),
    dict(q=P + 8), dict(out=P + 4), dict(lse=P + 2), dict(lengths=P + 1)])
def test_queries_that_are_refused(kw):
    assert refusal(cache(), None, attn(**kw))


@pytest.mark.parametrize("kw", [dict(lse=None), dict(scale=0.0), dict(max_len=1 << 30), dict(n_q_heads=8, q_stride=1024)])
def test_queries_that_are_taken(kw):
    assert refusal(cache(), None, attn(**kw)) is None
    assert refusal(cache(n_seqs=0, page_table=None), None, attn(q=None, out=None, lengths=None)) is None


def test_a_null_handle_is_refused():
    L = binding.lib()
    assert L.moss_enc_gemv_q4(None, P, P, P, P, P, 1, 16, 128, 0) == 1
    assert L.moss_enc_kv_append(None, ctypes.byref(cache()), ctypes.byref(rows())) == 1
    assert L.moss_enc_paged_attn(None, ctypes.byref(cache()), ctypes.byref(attn())) == 1
    assert L.moss_enc_paged_attn_workspace(None, ctypes.byref(cache()), 16, 0) == -1


def test_binding_refuses_tensors_that_are_no_cache():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(2, 2, dtype=torch.int32)
    for bad in [(k.float(), k.float(), t), (k, k.half(), t), (k[0], k[0], t), (k, k[:2], t), (k, k, t.long()), (k, k, t[0]),
                (k, k, t)]:  # the last: right, but not on a GPU
        with pytest.raises(ValueError):
            binding.KVCache(*bad)


def test_native_marshalling_refuses_what_is_not_on_the_gpu():
    m = binding.pycalls()  # loads without a GPU
    x = torch.zeros(1, 128, dtype=torch.bfloat16)
    codes, scales = torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(1, 16)
    for bad in [(x, codes, scales), (None, codes, scales), (1, codes, scales)]:
        with pytest.raises(ValueError):
            m.gemv_q4(0, 0, 0, *bad, None, None, 0)
    with pytest.raises(ValueError):
        m.gemv_q4(0, 0, 0)
    c = cache()
    k = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.kv_append(0, 0, 0, ctypes.addressof(c), k, k, i, None, None, None, None, False)
    with pytest.raises(ValueError):
        m.paged_attn(0, 0, 0, ctypes.addressof(c), k, i, None, None, None, False, 0, None)
    with pytest.raises(TypeError):
        m.gemv_q4("handle", 0, 0, x, codes, scales, None, None, 0)


class Calls:
    """Stands in for the native calls (and the library): records each."""

    def __init__(self, answer="done"):
        self.made, self.answer = [], answer

    def __getattr__(self, name):
        return lambda *a: (self.made.append((name, a)), self.answer)[1]


def encoder_on(device):
    """An Encoder without a handle, for what it does before and after a call."""
    e = object.__new__(binding.Encoder)
    e.h, e.hid, e.sid, e.device, e.torch = None, 0, 0, torch.device("cuda", device), torch
    return e


def test_a_cache_on_another_device_is_refused(monkeypatch):
    calls = Calls(-1)
    monkeypatch.setattr(binding, "pycalls", lambda: calls)
    monkeypatch.setattr(binding, "lib", lambda: calls)
    e = encoder_on(0)
    c = types.SimpleNamespace(device=torch.device("cuda", 1), address=P, ref=None)
    for call in (lambda: e.kv_append(c, None, None, None), lambda: e.paged_attn(c, None, None),
                 lambda: e.paged_attn_workspace(c, 8)):
        with pytest.raises(ValueError, match="device"):
            call()
    assert not calls.made


class Tensor:
    """Stands in for a tensor: which streams its memory was said to be used on."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


@pytest.mark.parametrize("same", [True, False])
def test_memory_on_its_way_is_not_handed_out_again(monkeypatch, same):
    # a handle on a stream of its own: what a call reads or writes may be freed
    # by the caller as soon as it returns (a temporary always is), and what it
    # made is used on the caller's stream
    mine, callers = "the handle's stream", "the caller's stream"
    e = encoder_on(0)
    e.sid, e.stream, e.current_stream = 7, mine, lambda device: 7 if same else 8
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: callers)
    made, lse = Tensor(), Tensor()
    c = types.SimpleNamespace(device=e.device, address=P, k=Tensor(), v=Tensor(), page_table=Tensor())
    pages = [c.k, c.v, c.page_table]

    def check(answer, call, n):
        calls = Calls(answer)
        monkeypatch.setattr(binding, "pycalls", lambda: calls)
        args = [Tensor() for _ in range(n)]
        assert call(*args) is answer and len(calls.made) == 1
        outs = [o for o in (answer if isinstance(answer, tuple) else (answer,)) if o is not None]
        assert all(t.streams == ([] if same else [mine]) for t in args + pages * (calls.made[0][0] != "gemv_q4"))
        assert all(t.streams == ([] if same else [callers]) for t in outs)
        for t in args + pages + outs:
            t.streams.clear()

    check(made, lambda x, q, s, b: e.gemv_q4(x, q, s, b), 4)
    check(made, lambda x, q, s, b, out: e.gemv_q4(x, q, s, b, out, 5), 5)
    check(None, lambda k, v, p: e.kv_append(c, k, v, p), 3)
    check(made, lambda k, v, p, s, q, o, i: e.kv_append(c, k, v, p, s, q, o, i, True), 7)
    check(made, lambda q, n: e.paged_attn(c, q, n), 2)
    check((made, lse), lambda q, n, o, l, w: e.paged_attn(c, q, n, None, o, l, True, 0, w), 5)
