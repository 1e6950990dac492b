"""What the cache and beam entry points refuse, on the host and before any GPU call (CPU only: every call here fails
validation or has nothing to do)."""

import ctypes

import pytest
import torch

import gated_deltanet_03_amd as gdn

NULL = ctypes.c_void_p(0)


def at(n):
    """An address that is never followed: 16-byte aligned, each far from the others."""
    return ctypes.c_void_p(0x100000000 * (n + 1))


@pytest.fixture(scope="module")
def lib():
    return gdn.load_library()


def last(lib):
    return lib.gdn_last_error().decode()


def cache(**kw):
    d = dict(N=2, T=5, Hq=8, Hkv=2, d=128, dtype=gdn.GDN_BF16, page_size=16, num_pages=40, max_pages=20)
    d.update(kw)
    return gdn.gdn_cache_shape(**d)


def append(lib, sh=None, how=None, **kw):
    sh = sh or cache()
    how = how or gdn.gdn_append_shape(sh.Hq * sh.d, sh.Hkv * sh.d, sh.Hkv * sh.d, 64, 0, 1)
    a = dict(q=at(0), k=at(1), v=at(2), freq=at(3), pos=NULL, axis=NULL, table=at(4), lens=at(5), cu=NULL, q_out=at(6),
             kc=at(7), vc=at(8))
    a.update(kw)
    return lib.gdn_cache_append(ctypes.byref(sh), ctypes.byref(how), *a.values(), NULL)


def attend(lib, sh=None, stride=None, scale=0.1, window=0, need=None, **kw):
    sh = sh or cache()
    a = dict(kc=at(7), vc=at(8), table=at(4), lens=at(5), cu=NULL)
    a.update({n: kw.pop(n) for n in list(kw) if n in a})
    b = dict(q=at(0), o=at(6), ws=at(9), n=1 << 40)
    b.update(kw)
    return lib.gdn_cache_attention(ctypes.byref(sh), b["q"], stride or sh.Hq * sh.d, *a.values(), scale, window, b["o"],
                                   b["ws"], b["n"], NULL)


INVALID, UNSUPPORTED, OK = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_OK


@pytest.mark.parametrize("kw,status,word", [
    (dict(N=-1), INVALID, "N=-1"), (dict(T=-1), INVALID, "T=-1"), (dict(Hq=7), INVALID, "multiple"),
    (dict(Hkv=0), INVALID, "multiple"), (dict(dtype=9), INVALID, "gdn_dtype"), (dict(d=16), UNSUPPORTED, "d=16"),
    (dict(d=96), UNSUPPORTED, "d=96"), (dict(page_size=0), INVALID, "page_size"),
    (dict(page_size=24), UNSUPPORTED, "page_size=24"), (dict(page_size=2048), UNSUPPORTED, "page_size"),
    (dict(max_pages=(1 << 22) + 1), UNSUPPORTED, "2^26"), (dict(num_pages=1 << 27), UNSUPPORTED, "rows"),
    (dict(N=1 << 20, T=1 << 11), UNSUPPORTED, "tokens"), (dict(num_pages=-1), INVALID, "num_pages"),
])
def test_cache_shapes(lib, kw, status, word):
    for call in (append, attend):
        assert call(lib, cache(**kw)) == status and word in last(lib)
    sh = cache(**kw)
    with pytest.raises(gdn.GdnError, match="."):
        gdn.gdn_cache_attention_workspace_bytes(sh, False)


def test_append_refusals(lib):
    def how(q=1024, k=256, v=256, rotary=64, axes=1):
        return gdn.gdn_append_shape(q, k, v, rotary, 0, axes)
    for h, word in ((how(rotary=3), "rotary"), (how(rotary=130), "rotary"), (how(rotary=-2), "rotary"),
                    (how(axes=0), "axes"), (how(axes=9), "axes"), (how(q=1020), "q_token_stride"),
                    (how(k=128), "k_token_stride"), (how(v=257), "v_token_stride"), (how(k=1 << 33), "k_token_stride"),
                    (how(axes=2), "positions"), (how(rotary=0), "inv_freq")):
        assert append(lib, how=h) == INVALID and word in last(lib), word
    for kw, word in ((dict(k=NULL), "k is NULL"), (dict(v=NULL), "v is NULL"), (dict(q_out=NULL), "together"),
                     (dict(q=NULL), "together"), (dict(freq=NULL), "inv_freq"), (dict(kc=NULL), "k_cache"),
                     (dict(lens=NULL), "cache_lens"), (dict(table=NULL), "block_table"),
                     (dict(k=ctypes.c_void_p(0x200000008)), "aligned"), (dict(vc=ctypes.c_void_p(0x200000008)), "aligned"),
                     (dict(lens=ctypes.c_void_p(0x200000002)), "aligned"), (dict(pos=ctypes.c_void_p(0x200000002)), "aligned"),
                     (dict(q_out=ctypes.c_void_p(0x200000008)), "aligned"),
                     (dict(kc=at(1)), "overlaps"), (dict(vc=at(7)), "overlaps"), (dict(q_out=at(1)), "overlaps"),
                     (dict(q_out=at(8)), "overlaps"), (dict(kc=at(4)), "overlaps"), (dict(q_out=at(5)), "overlaps")):
        assert append(lib, **kw) == INVALID and word in last(lib), (kw, last(lib))
    # in place only where q is contiguous
    assert append(lib, how=how(q=2048), q_out=at(0)) == INVALID and "overlaps" in last(lib)
    assert append(lib, cache(N=0)) == OK and append(lib, cache(T=0)) == OK


def test_attention_refusals(lib):
    for kw, word in ((dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"),
                     (dict(scale=float("inf")), "scale"), (dict(window=-1), "window"), (dict(stride=1023), "stride"),
                     (dict(stride=512), "stride"), (dict(q=NULL), "q is NULL"), (dict(o=NULL), "o is NULL"),
                     (dict(kc=NULL), "k_cache"), (dict(table=NULL), "block_table"), (dict(lens=NULL), "cache_lens"),
                     (dict(o=ctypes.c_void_p(0x200000008)), "aligned"), (dict(o=at(0)), "overlaps"),
                     (dict(o=at(8)), "overlaps")):
        assert attend(lib, **kw) == INVALID and word in last(lib), (kw, last(lib))
    wide = cache(max_pages=100)               # sequences that may be cut: a workspace
    assert gdn.gdn_cache_attention_workspace_bytes(wide, False) > 64
    for kw, word in ((dict(ws=NULL), "workspace"), (dict(n=64), "workspace"), (dict(ws=at(6)), "overlaps"),
                     (dict(ws=ctypes.c_void_p(0x200000008)), "aligned"), (dict(ws=at(7)), "overlaps")):
        assert attend(lib, wide, **kw) == INVALID and word in last(lib), (kw, last(lib))
    assert attend(lib, cache(N=0)) == OK and attend(lib, cache(T=0)) == OK
    assert gdn.gdn_cache_attention_workspace_bytes(cache(N=0), False) == 0
    assert gdn.gdn_cache_attention_workspace_bytes(cache(max_pages=1), False) == 0      # one page: nothing to split


def beam(lib, sh=None, **kw):
    s = dict(B=2, W=4, K=4, V=1000, dtype=gdn.GDN_F32, eos_token=-1, pad_token=0, row_stride=1000)
    s.update(sh or {})
    a = dict(x=at(0), scores=at(1), finished=NULL, tokens=at(2), parents=at(3), new_scores=at(4), new_finished=at(5),
             ws=at(6), n=1 << 40)
    a.update(kw)
    return lib.gdn_beam_select(ctypes.byref(gdn.gdn_beam_shape(**s)), *a.values(), NULL)


def test_beam_refusals(lib):
    for sh, status, word in ((dict(B=-1), INVALID, "B=-1"), (dict(W=0), INVALID, "W=0"), (dict(K=0), INVALID, "K=0"),
                             (dict(V=0), INVALID, "V=0"), (dict(dtype=5), INVALID, "gdn_dtype"),
                             (dict(row_stride=999), INVALID, "row_stride"), (dict(pad_token=1000), INVALID, "pad_token"),
                             (dict(pad_token=-1), INVALID, "pad_token"), (dict(W=65), UNSUPPORTED, "64"),
                             (dict(K=65), UNSUPPORTED, "64"), (dict(V=(1 << 24) + 1, row_stride=1 << 25), UNSUPPORTED, "2^24"),
                             (dict(B=(1 << 20) + 1), UNSUPPORTED, "2^20")):
        assert beam(lib, sh) == status and word in last(lib), sh
    for kw, word in ((dict(x=NULL), "required"), (dict(tokens=NULL), "required"), (dict(new_finished=NULL), "required"),
                     (dict(x=ctypes.c_void_p(0x200000002)), "aligned"), (dict(parents=ctypes.c_void_p(0x200000002)), "aligned"),
                     (dict(ws=NULL), "workspace"), (dict(n=100), "workspace"), (dict(ws=ctypes.c_void_p(0x200000008)), "aligned"),
                     (dict(new_scores=at(1)), "overlaps"), (dict(tokens=at(0)), "overlaps"), (dict(parents=at(2)), "overlaps"),
                     (dict(finished=at(8), new_finished=at(8)), "overlaps"), (dict(ws=at(0)), "overlaps")):
        assert beam(lib, **kw) == INVALID and word in last(lib), (kw, last(lib))
    assert beam(lib, dict(B=0)) == OK
    with pytest.raises(gdn.GdnError, match="64"):
        gdn.gdn_beam_workspace_bytes(gdn.gdn_beam_shape(1, 65, 1, 10, 0, -1, 0, 10))


def reorder(lib, sh=None, src=at(0), dst=at(1), si=at(2), di=NULL):
    s = dict(layers=2, src_layer_stride=1 << 20, dst_layer_stride=1 << 20, src_rows=8, dst_rows=8, row_bytes=1024,
             src_group=4, G=2, W=4)
    s.update(sh or {})
    return lib.gdn_state_reorder(ctypes.byref(gdn.gdn_reorder_shape(**s)), src, dst, si, di, NULL)


def test_reorder_refusals(lib):
    for sh, status, word in ((dict(layers=-1), INVALID, ">= 0"), (dict(row_bytes=24), INVALID, "multiples of 16"),
                             (dict(src_layer_stride=8), INVALID, "multiples of 16"), (dict(W=65), UNSUPPORTED, "64"),
                             (dict(row_bytes=1 << 41), UNSUPPORTED, "2^46"), (dict(src_rows=1 << 40), UNSUPPORTED, "2^46"),
                             (dict(dst_layer_stride=4096), INVALID, "smaller than a layer"),
                             (dict(layers=1 << 39, src_layer_stride=1 << 30), UNSUPPORTED, "2^62")):
        assert reorder(lib, sh) == status and word in last(lib), (sh, last(lib))
    for kw, word in ((dict(src=NULL), "required"), (dict(dst=NULL), "required"), (dict(si=NULL), "required"),
                     (dict(src=ctypes.c_void_p(0x200000008)), "aligned"), (dict(si=ctypes.c_void_p(0x200000002)), "aligned"),
                     (dict(dst=ctypes.c_void_p(at(0).value + 1024)), "overlaps"), (dict(si=at(1)), "overlaps"),
                     (dict(di=ctypes.c_void_p(at(1).value + (1 << 20))), "overlaps")):
        assert reorder(lib, **kw) == INVALID and word in last(lib), (kw, last(lib))
    assert reorder(lib, dict(src_layer_stride=1 << 21), dst=at(0)) == INVALID and "equal" in last(lib)
    for zero in ("layers", "G", "W", "row_bytes", "src_rows", "dst_rows"):
        assert reorder(lib, {zero: 0}) == OK


# ---------------------------------------------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------------------------------------------
def tensors(**kw):
    bf = torch.bfloat16
    t = dict(q=torch.zeros(3, 8, 64, dtype=bf), k=torch.zeros(3, 2, 64, dtype=bf), v=torch.zeros(3, 2, 64, dtype=bf),
             kc=torch.zeros(5, 2, 16, 64, dtype=bf), vc=torch.zeros(5, 2, 16, 64, dtype=bf),
             table=torch.zeros(2, 2, dtype=torch.int32), lens=torch.zeros(2, dtype=torch.int32),
             cu=torch.zeros(3, dtype=torch.int32), freq=torch.zeros(32))
    t.update(kw)
    return t


def call_append(t, **kw):
    return gdn.gdn_cache_append(t["k"], t["v"], t["kc"], t["vc"], t["table"], t["lens"],
                                **{**dict(cu_seqlens=t["cu"], q=t["q"], inv_freq=t["freq"]), **kw})


def call_attend(t, **kw):
    return gdn.gdn_cache_attention(t["q"], t["kc"], t["vc"], t["table"], t["lens"], **{**dict(cu_seqlens=t["cu"]), **kw})


def test_binding_wants_a_gpu():
    for call in (call_append, call_attend):
        with pytest.raises(ValueError, match="GPU"):
            call(tensors())


@pytest.mark.parametrize("kw,error,word", [
    (dict(kc=torch.zeros(5, 2, 16, 64, dtype=torch.float64)), TypeError, "unsupported"),
    (dict(vc=torch.zeros(5, 2, 16, 32, dtype=torch.bfloat16)), ValueError, "v_cache"),
    (dict(vc=torch.zeros(5, 2, 16, 64)), TypeError, "v_cache"),
    (dict(kc=torch.zeros(5, 2, 16, 128, dtype=torch.bfloat16)[..., :64]), ValueError, "contiguous"),
    (dict(table=torch.zeros(2, 2)), TypeError, "block_table"), (dict(table=torch.zeros(2, dtype=torch.int32)), ValueError, "block_table"),
    (dict(lens=torch.zeros(3, dtype=torch.int32)), ValueError, "cache_lens"),
    (dict(lens=torch.zeros(2, dtype=torch.int64)), TypeError, "cache_lens"),
    (dict(cu=torch.zeros(2, dtype=torch.int32)), ValueError, "cu_seqlens"),
    (dict(q=torch.zeros(3, 7, 64, dtype=torch.bfloat16)), ValueError, "multiple"),
    (dict(q=torch.zeros(3, 8, 32, dtype=torch.bfloat16)), ValueError, "q has shape"),
    (dict(q=torch.zeros(3, 8, 64)), TypeError, "q must be"), (dict(q=torch.zeros(3, 512, dtype=torch.bfloat16)), ValueError, "q must be"),
    (dict(q=torch.zeros(3, 64, 8, dtype=torch.bfloat16).transpose(1, 2)), ValueError, "contiguous within a token"),
    (dict(q=torch.zeros(1, 8, 64, dtype=torch.bfloat16).expand(3, 8, 64)), ValueError, "overlap"),
])
def test_binding_refusals(kw, error, word):
    for call in (call_append, call_attend):
        with pytest.raises(error, match=word):
            call(tensors(**kw))


def test_binding_append_refusals():
    t = tensors()
    i32 = torch.int32
    for kw, error, word in ((dict(inv_freq=None), ValueError, "without inv_freq"), (dict(q=None, q_out=t["q"]), ValueError, "without q"),
                            (dict(inv_freq=torch.zeros(33)), ValueError, "rotary"), (dict(inv_freq=torch.zeros(0)), ValueError, "rotary"),
                            (dict(positions=torch.zeros(4, dtype=i32)), ValueError, "positions"),
                            (dict(positions=torch.zeros(2, 3, dtype=i32)), ValueError, "pair_axis"),
                            (dict(positions=torch.zeros(3)), TypeError, "positions"),
                            (dict(pair_axis=torch.zeros(31, dtype=i32)), ValueError, "pair_axis"),
                            (dict(q_out=torch.zeros(2, 8, 64, dtype=torch.bfloat16)), ValueError, "q_out")):
        with pytest.raises(error, match=word):
            call_append(t, **kw)
    with pytest.raises(ValueError, match="2 sequences"):
        call_append(tensors(v=torch.zeros(4, 2, 64, dtype=torch.bfloat16)))
    dense = tensors(k=torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16), v=torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16),
                    q=torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="q has shape"):
        call_append(dense, cu_seqlens=None)
    uneven = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)[:, :3]
    with pytest.raises(ValueError, match="evenly"):
        call_append(tensors(k=uneven, v=dense["v"]), cu_seqlens=None, q=None, inv_freq=None)
    with pytest.raises(ValueError, match="3 sequences"):
        call_attend(tensors(q=torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16), table=torch.zeros(3, 2, dtype=i32),
                            lens=torch.zeros(3, dtype=i32)), cu_seqlens=None)


def test_binding_beam_refusals():
    x, s = torch.zeros(2, 3, 10), torch.zeros(2, 3)
    for a, kw, error, word in (((x[0], s), {}, ValueError, "B, W, V"), ((x.double(), s), {}, TypeError, "unsupported"),
                               ((x, s[:1]), {}, ValueError, "scores"), ((x, s.double()), {}, TypeError, "scores"),
                               ((x, s), dict(finished=torch.zeros(2, 3)), TypeError, "finished"), ((x, s), dict(beams=0), ValueError, "beams"),
                               ((x, s), dict(tokens=torch.zeros(2, 4, dtype=torch.int32)), ValueError, "tokens"),
                               ((x, s), dict(eos_token=1 << 31), ValueError, "eos_token"), ((x, s), {}, ValueError, "GPU"),
                               ((x.transpose(1, 2), torch.zeros(2, 10)), {}, ValueError, "vocabulary")):
        with pytest.raises(error, match=word):
            gdn.gdn_beam_select(*a, **kw)


def test_binding_reorder_refusals():
    s, p = torch.zeros(6, 8), torch.zeros(2, 3, dtype=torch.int32)
    for a, kw, error, word in (((s, p[0]), {}, ValueError, "B, K"), ((s, p.long()), {}, TypeError, "parents"),
                               ((s[:5], p), {}, ValueError, "5 rows"), ((s, p), dict(axis=2), ValueError, "axis"),
                               ((s, p[:, :2].contiguous()), dict(out=s), ValueError, "out has shape"),
                               ((s[:, :7].contiguous(), p), {}, ValueError, "multiple of 16"), ((s, p), dict(out=s), ValueError, "GPU"),
                               ((s.t(), p), {}, ValueError, "contiguous")):
        with pytest.raises(error, match=word):
            gdn.gdn_state_reorder(*a, **kw)
    c = torch.zeros(4, 1, 16, 32)
    for a, error, word in (((c, c[:3], p, p), ValueError, "one shape"), ((c, c, p, p[:1]), ValueError, "src_pages"),
                           ((c, c, p.long(), p), TypeError, "src_pages"), ((c, c.clone(), p, p), ValueError, "GPU")):
        with pytest.raises(error, match=word):
            gdn.gdn_cache_copy_pages(*a)


@pytest.mark.parametrize("window", [-1, 1 << 31, 1 << 40])
def test_binding_window(window):
    with pytest.raises(ValueError, match="window"):
        call_attend(tensors(), window=window)


def test_launches_on_the_tensors_device(monkeypatch):
    """A kernel starts on the current device; tensors of another one make that current for the call."""
    seen, entered = [], []

    class Device:
        def __init__(self, dev):
            entered.append(dev)

        def __enter__(self):
            seen.append("in")

        def __exit__(self, *a):
            seen.append("out")
    monkeypatch.setattr(gdn, "_on_gpu", lambda dev: 1000 + dev.index)
    monkeypatch.setattr(gdn, "_current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", Device)
    for index in (1, 0):
        gdn._launch(torch.device("cuda", index), lambda *a: seen.append(a), "x")
    assert seen == [("x", 1001), "in", ("x", 1000), "out"] and entered == [torch.device("cuda", 0)]
    with pytest.raises(gdn.GdnError):
        gdn._launch(torch.device("cuda", 0), lambda *a: gdn.GDN_ERR_INVALID_ARG)


def test_scales_beyond_the_largest_float(lib):
    """scale is applied times log2(e) in fp32, which has to be finite too; the largest and smallest that are pass."""
    top = 2.0 ** 128 * (1 - 2.0 ** -24)
    for scale in (top, 0.99 * top, top / 1.44):
        assert attend(lib, scale=scale) == INVALID and "scale" in last(lib), scale
    for scale in (top / 1.4427, 1e-45):
        assert attend(lib, scale=scale, q=NULL) == INVALID and "q is NULL" in last(lib), scale
