"""Refusals of the linear attention, the draft verification and the block norms,
in the binding (CPU tensors, before any library call) and at the C ABI (fake
pointers that fail validation before any HIP call)."""

import ctypes

import pytest
import torch

import gated_deltanet_03_amd as gdn

A = [ctypes.c_void_p(0x10000000 * i) for i in range(1, 14)]   # far apart, never dereferenced
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    return gdn.load_library()


def last(lib):
    return lib.gdn_last_error().decode()


def tokens(T=20, Hq=2, Hv=4, dk=16, dv=32):
    return (torch.zeros(T, Hq, dk), torch.zeros(T, Hq, dk), torch.zeros(T, Hv, dv), torch.zeros(T, Hv),
            torch.tensor([0, 7, T], dtype=torch.int32))


@pytest.mark.parametrize("call", ["gdn_linear_prefill", "gdn_linear_step"])
def test_linear_binding(call):
    f = getattr(gdn, call)
    q, k, v, g, cu = tokens()
    with pytest.raises(ValueError, match="k has shape"):
        f(q, k[:-1], v, g, cu_seqlens=cu)
    with pytest.raises(ValueError, match="v has shape"):
        f(q, k, v[1:], g, cu_seqlens=cu)
    with pytest.raises(ValueError, match="g has shape"):
        f(q, k, v, g[:, :3].contiguous(), cu_seqlens=cu)
    with pytest.raises(ValueError, match="g has shape"):
        f(q, k, v, g[0, :2].contiguous(), cu_seqlens=cu)
    with pytest.raises(TypeError, match="g must be"):
        f(q, k, v, g.half(), cu_seqlens=cu)
    with pytest.raises(TypeError, match="v must be"):
        f(q, k, v.half(), g, cu_seqlens=cu)
    with pytest.raises(TypeError, match="cu_seqlens must be"):
        f(q, k, v, g, cu_seqlens=cu.long())
    with pytest.raises(ValueError, match="contiguous"):
        f(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, g, cu_seqlens=cu)
    with pytest.raises(ValueError, match="o has shape"):
        f(q, k, v, g, cu_seqlens=cu, o=torch.zeros(20, 4, 16))
    with pytest.raises(ValueError, match="final_state has shape"):
        f(q, k, v, g, cu_seqlens=cu, final_state=torch.zeros(3, 4, 16, 32))
    with pytest.raises(ValueError, match="initial_state has"):
        f(q, k, v, g, cu_seqlens=torch.tensor([0, 3, 7, 20], dtype=torch.int32), initial_state=torch.zeros(2, 4, 16, 32))
    with pytest.raises(ValueError, match="multiple"):
        f(q, k, torch.zeros(20, 3, 32), torch.zeros(20, 3), cu_seqlens=cu)
    with pytest.raises(ValueError, match="expected a GPU"):
        f(q, k, v, g, cu_seqlens=cu)


def test_linear_step_capture_binding():
    q, k, v, g, cu = tokens()
    with pytest.raises(ValueError, match="capture_count is required"):
        gdn.gdn_linear_step(q, k, v, g, cu_seqlens=cu, state_update_capacity=2)
    with pytest.raises(ValueError, match="capture_count has"):
        gdn.gdn_linear_step(q, k, v, g, cu_seqlens=cu, state_update_capacity=2,
                            capture_count=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="state_update has"):
        gdn.gdn_linear_step(q, k, v, g, cu_seqlens=cu, state_update_capacity=2,
                            capture_count=torch.zeros(2, dtype=torch.int32), state_update=torch.zeros(2, 1, 164))


def test_verify_binding():
    p, q = torch.zeros(2, 4, 9), torch.zeros(2, 3, 9)
    x, u = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 4)
    f = gdn.gdn_verify_drafts
    with pytest.raises(ValueError, match="target_probs has shape"):
        f(p[:, :3], q, x, u)
    with pytest.raises(ValueError, match="draft_probs has shape"):
        f(p, q[:, :, :8], x, u)
    with pytest.raises(TypeError, match="draft_probs must be"):
        f(p, q.half(), x, u)
    with pytest.raises(TypeError, match="draft_tokens must be"):
        f(p, q, x.long(), u)
    with pytest.raises(ValueError, match="uniforms has"):
        f(p, q, x, u[:, :3].contiguous())
    with pytest.raises(ValueError, match="draft_count has"):
        f(p, q, x, u, draft_count=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="tokens has"):
        f(p, q, x, u, tokens=torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="along the vocabulary"):
        f(torch.zeros(2, 4, 18)[:, :, ::2], q, x, u)
    with pytest.raises(ValueError, match="evenly spaced"):
        f(torch.zeros(2, 5, 9)[:, :4], q, x, u)
    with pytest.raises(ValueError, match="evenly spaced"):
        f(torch.zeros(1, 1, 9).expand(2, 4, 9), q, x, u)
    with pytest.raises(ValueError, match="expected a GPU"):
        f(p, q, x, u)


def test_norm_binding():
    y = torch.zeros(3, 48)
    f = gdn.gdn_block_norm
    with pytest.raises(ValueError, match="gate has shape"):
        f(y, gate=torch.zeros(3, 47))
    with pytest.raises(TypeError, match="residual must be"):
        f(y, residual=y.half())
    with pytest.raises(ValueError, match="gate_act"):
        f(y, gate=y, gate_act="relu")
    with pytest.raises(ValueError, match="gate_act 'none'"):
        f(y, gate=y, gate_act="none")
    with pytest.raises(ValueError, match="divisor"):
        f(y, post_weight=torch.zeros(32))
    with pytest.raises(ValueError, match="next_weight has"):
        f(y, next_weight=torch.zeros(47))
    with pytest.raises(ValueError, match="without next_weight"):
        f(y, normed=torch.zeros(3, 48))
    with pytest.raises(ValueError, match="contiguous"):
        f(torch.zeros(3, 96)[:, ::2])
    with pytest.raises(ValueError, match="expected a GPU"):
        f(y)


def shape(**kw):
    d = dict(B=2, T=64, Hq=2, Hv=4, dk=128, dv=128, scale=0.088, dtype=gdn.GDN_BF16)
    d.update(kw)
    return gdn.gdn_shape(**d)


def prefill(lib, sh, q=A[0], k=A[1], v=A[2], g=A[3], gs=4, s0=NULL, stride=0, cu=NULL, o=A[4], so=NULL, ws=NULL, n=0):
    return lib.gdn_linear_prefill(ctypes.byref(sh), q, k, v, g, gs, s0, stride, cu, o, so, ws, n, NULL)


def step(lib, sh, q=A[0], k=A[1], v=A[2], g=A[3], gs=4, s0=NULL, stride=0, cu=NULL, o=A[4], so=NULL, cap=0,
         counts=NULL, su=NULL):
    return lib.gdn_linear_step(ctypes.byref(sh), q, k, v, g, gs, s0, stride, cu, o, so, cap, counts, su, NULL)


def test_linear_abi(lib):
    bad, uns = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED
    per = 4 * 128 * 128
    for call in (prefill, step):
        assert call(lib, shape(Hv=5)) == bad and "multiple" in last(lib)
        assert call(lib, shape(dk=48)) == uns
        assert call(lib, shape(B=1, T=(1 << 30) + 1)) == uns and "2^30" in last(lib)
        assert call(lib, shape(dtype=5)) == bad
        assert call(lib, shape(), gs=3) == bad and "g_token_stride" in last(lib)
        assert call(lib, shape(), k=NULL) == bad and "k is NULL" in last(lib)
        assert call(lib, shape(), v=ctypes.c_void_p(0x30000008)) == bad and "aligned" in last(lib)
        assert call(lib, shape(), o=A[2]) == bad and "o overlaps v" in last(lib)
        assert call(lib, shape(), so=A[3]) == bad and "final_state overlaps g" in last(lib)
        assert call(lib, shape(), s0=A[5], stride=0, so=A[5]) == bad and "in-place" in last(lib)
        assert call(lib, shape(), s0=A[5], stride=per + 2) == bad
        assert call(lib, shape(), s0=A[4], stride=per) == bad and "o overlaps initial_state" in last(lib)
    assert step(lib, shape(), cap=-1) == bad
    assert step(lib, shape(), cap=1, su=A[6]) == bad and "capture_count" in last(lib)
    assert step(lib, shape(), cap=1, counts=A[6]) == bad and "state_update" in last(lib)
    assert step(lib, shape(), cap=1, counts=A[6], su=A[0]) == bad and "overlaps q" in last(lib)
    assert step(lib, shape(), cap=1, counts=A[4], su=A[6]) == bad and "capture_count" in last(lib)


def test_linear_workspace(lib):
    assert gdn.gdn_linear_workspace_bytes(shape(), False) == 0                       # short rows
    assert gdn.gdn_linear_workspace_bytes(shape(B=64, Hv=32, T=4096), False) == 0    # many rows
    long = shape(B=1, T=8192)
    need = gdn.gdn_linear_workspace_bytes(long, False)
    assert need > 0 and prefill(lib, long) == gdn.GDN_ERR_INVALID_ARG and "workspace" in last(lib)
    assert prefill(lib, long, ws=A[6], n=need - 1) == gdn.GDN_ERR_INVALID_ARG
    assert prefill(lib, long, ws=ctypes.c_void_p(0x70000008), n=need) == gdn.GDN_ERR_INVALID_ARG
    assert prefill(lib, long, ws=A[1], n=need) == gdn.GDN_ERR_INVALID_ARG and "workspace overlaps k" in last(lib)
    with pytest.raises(gdn.GdnError, match="2\\^30"):
        gdn.gdn_linear_workspace_bytes(shape(B=3, T=1 << 29), False)
    with pytest.raises(gdn.GdnError, match="supported head dims"):
        gdn.gdn_linear_workspace_bytes(shape(dk=40), False)


def test_verify_abi(lib):
    bad, uns = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED

    def call(B=2, K=3, V=1000, dtype=gdn.GDN_F32, ps=1000, qs=1000, p=A[0], q=A[1], x=A[2], u=A[3], n=NULL, t=A[4],
             e=A[5], ws=A[6], wsb=1 << 20):
        sh = gdn.gdn_verify_shape(B, K, V, dtype, ps, qs)
        return lib.gdn_verify_drafts(ctypes.byref(sh), p, q, x, u, n, t, e, ws, wsb, NULL)
    assert call(V=0) == bad and call(B=-1) == bad and call(K=-1) == bad and call(dtype=3) == bad
    assert call(ps=999) == bad and "row strides" in last(lib)
    assert call(V=1 << 25, ps=1 << 25, qs=1 << 25) == uns
    assert call(p=NULL) == bad and call(x=NULL) == bad and call(t=NULL) == bad
    assert call(p=ctypes.c_void_p(0x10000002)) == bad and "aligned" in last(lib)
    long = dict(V=100000, ps=100000, qs=100000)
    assert call(ws=NULL, **long) == bad and call(wsb=8, **long) == bad and "workspace" in last(lib)
    assert call(t=A[3]) == bad and "tokens overlaps uniforms" in last(lib)
    assert call(e=A[4]) == bad and "emit_count overlaps tokens" in last(lib)
    assert call(ws=A[0], **long) == bad and "workspace overlaps target_probs" in last(lib)


def test_norm_abi(lib):
    bad, uns = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED

    def call(T=4, D=256, group=256, dtype=gdn.GDN_BF16, act=0, scale=1.0, eps=1e-6, y=A[0], gate=NULL, res=NULL,
             wp=NULL, wn=NULL, h=A[1], n=NULL):
        sh = gdn.gdn_norm_shape(T, D, group, dtype, act, scale, eps)
        return lib.gdn_block_norm(ctypes.byref(sh), y, gate, res, wp, wn, h, n, NULL)
    assert call(D=0) == bad and call(T=-1) == bad and call(dtype=9) == bad and call(act=3, gate=A[2]) == bad
    assert call(group=100) == bad and call(group=8) == uns and call(D=16385, group=16385) == uns
    assert call(eps=-1.0) == bad and call(eps=float("nan")) == bad and call(scale=float("nan")) == bad
    assert call(act=1) == bad and call(gate=A[2]) == bad and "gate" in last(lib)
    assert call(wn=A[2]) == bad and call(n=A[2]) == bad and "together" in last(lib)
    assert call(y=NULL) == bad and call(h=NULL) == bad
    assert call(h=ctypes.c_void_p(0x20000001)) == bad and "aligned" in last(lib)
    assert call(act=1, gate=A[1]) == bad and "h overlaps gate" in last(lib)
    assert call(h=ctypes.c_void_p(0x10000010)) == bad and "h overlaps y" in last(lib)
    assert call(wn=A[2], n=A[0]) == bad and "normed overlaps y" in last(lib)
    assert call(wn=A[2], n=A[1]) == bad and "normed overlaps h" in last(lib)


def test_sizes_beyond_32_bits_are_refused():
    """The C structs hold 32-bit sizes: a larger one must not be cut to its low bits."""
    def n(*s, dtype=torch.bfloat16):
        return torch.empty(*s, dtype=dtype, device="meta")
    big = 2 ** 32 + 32
    with pytest.raises(ValueError, match="V=4294967328 does not fit 32 bits"):
        gdn.gdn_verify_drafts(n(1, 1, big), None, n(1, 0, dtype=torch.int32), n(1, 1, dtype=torch.float32))
    with pytest.raises(ValueError, match="D=4294967328 does not fit 32 bits"):
        gdn.gdn_block_norm(n(1, big))
    for call in (gdn.gdn_linear_prefill, gdn.gdn_linear_step):
        with pytest.raises(ValueError, match="T=4294967328 does not fit 32 bits"):
            call(n(1, big, 1, 16), n(1, big, 1, 16), n(1, big, 1, 16), n(1, dtype=torch.float32))
