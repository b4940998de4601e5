"""Refusals of the decode-step operators on the host (CPU only): the C entry points with placeholder
addresses that are never used, and the tensor wrappers."""

import pytest
import torch

from adapter_lora_projection_amd import _lib, decode_ops as d, ops

bf = torch.bfloat16
OK, EINVAL, EUNSUP, EWS = _lib.LORA_OK, _lib.LORA_EINVAL, _lib.LORA_EUNSUPPORTED, _lib.LORA_EWORKSPACE
nan, inf = float("nan"), float("inf")


def _prep(**kw):
    a = dict(dtype=1, K=256, N=32, group=64, codes=0x1000, ldc=128, scales=0x2000, lds=4, zeros=0x3000, ldz=4,
             prepared=0x4000, nbytes=1 << 20, stream=None)
    a.update(kw)
    return _lib.lib().lora_linear_w4_prepare(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), EUNSUP), (dict(dtype=5), EUNSUP), (dict(K=0), EINVAL), (dict(N=0), EINVAL),
    (dict(group=0), EINVAL), (dict(group=48), EUNSUP), (dict(group=256), EUNSUP), (dict(K=96), EINVAL),
    (dict(K=1 << 25), EUNSUP), (dict(N=1 << 25), EUNSUP), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(prepared=None), EINVAL), (dict(ldc=127), EINVAL), (dict(lds=3), EINVAL), (dict(ldz=3), EINVAL),
    (dict(prepared=0x4008), EUNSUP), (dict(nbytes=4096), EWS),
])
def test_w4_prepare_refusals(kw, code):
    assert _prep(**kw) == code


def _w4(**kw):
    a = dict(dtype=1, M=4, K=256, N=32, group=64, zp=0, x=0x1000, ldx=256, w=0x2000, y=0x3000, ldy=32,
             ws=None, nbytes=0, stream=None)
    a.update(kw)
    return _lib.lib().lora_linear_w4(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), EUNSUP), (dict(M=-1), EINVAL), (dict(M=(1 << 19) + 1), EUNSUP), (dict(K=250), EINVAL),
    (dict(group=16), EUNSUP), (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(y=None), EINVAL),
    (dict(ldx=255), EINVAL), (dict(ldx=260), EUNSUP), (dict(ldy=31), EINVAL), (dict(x=0x1002), EUNSUP),
    (dict(w=0x2008), EUNSUP), (dict(M=0, x=None, y=None), OK),
    (dict(M=64, K=8192, N=4096, group=128, ldx=8192, ldy=4096), EWS),  # needs planes
    (dict(M=64, K=8192, N=4096, group=128, ldx=8192, ldy=4096, ws=0x10008, nbytes=1 << 40), EWS),
])
def test_w4_refusals(kw, code):
    assert _w4(**kw) == code


def test_w4_prepared_size():
    # 2 x 2 tiles of 1 KiB, 2 x 4 groups of 16 scales of 2 bytes (4 with zero points)
    assert _lib.lora_linear_w4_prepared_size(1, 256, 32, 64, 0) == 4096 + 256
    assert _lib.lora_linear_w4_prepared_size(1, 256, 32, 64, 1) == 4096 + 512
    assert _lib.lora_linear_w4_prepared_size(1, 96, 17, 32, 0) == 2048 + 256  # 192 rounded up to 256
    assert _lib.lora_linear_w4_prepared_size(0, 256, 32, 64, 0) == 0
    assert _lib.lora_linear_w4_prepared_size(1, 250, 32, 64, 0) == 0


def test_w4_workspace_size():
    size = _lib.lora_linear_w4_workspace_size
    assert size(1, 1, 16384, 28672, 128) == 0 and size(1, 2, 16384, 1024, 128) == 0
    n = size(1, 64, 8192, 4096, 128)  # planes of [64][4096] floats
    assert n > 0 and n % (64 * 4096 * 4) == 0
    assert size(1, 0, 8192, 4096, 128) == 0 and size(1, 64, 8192, 4096, 48) == 0 and size(0, 64, 8192, 4096, 128) == 0


def _rope(**kw):
    a = dict(dtype=1, T=4, Hq=4, Hkv=2, D=64, rot=64, inter=0, pages=8, page=16, rows=100, q=0x1000, ldq=256,
             k=0x2000, ldk=128, v=0x3000, ldv=128, table=0x4000, positions=0x5000, slots=0x6000, qn=None, kn=None,
             eps=1e-6, qo=0x7000, ldqo=256, kc=0x8000, vc=0x9000, ps=16 * 128, ts=128, hs=64, stream=None)
    a.update(kw)
    return _lib.lib().lora_rope_append(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), EUNSUP), (dict(T=-1), EINVAL), (dict(Hq=-1), EINVAL), (dict(Hkv=0), EINVAL), (dict(D=0), EINVAL),
    (dict(D=1025, rot=64), EUNSUP), (dict(rot=0), EINVAL), (dict(rot=63), EINVAL), (dict(rot=66), EINVAL),
    (dict(pages=-1), EINVAL), (dict(page=0), EINVAL), (dict(rows=0), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=nan), EINVAL), (dict(T=1 << 28), EUNSUP), (dict(q=None), EINVAL), (dict(qo=None), EINVAL),
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(table=None), EINVAL), (dict(positions=None), EINVAL),
    (dict(slots=None), EINVAL), (dict(kc=None), EINVAL), (dict(vc=None), EINVAL), (dict(ldq=255), EINVAL),
    (dict(ldqo=255), EINVAL), (dict(ldk=127), EINVAL), (dict(ldv=127), EINVAL), (dict(ps=-1), EINVAL),
    (dict(ts=-128), EINVAL), (dict(hs=-64), EINVAL), (dict(hs=63), EINVAL), (dict(ts=64), EINVAL),
    (dict(ps=0), EINVAL), (dict(ps=15 * 128), EINVAL), (dict(T=0, q=None, k=None, kc=None), OK),
])
def test_rope_refusals(kw, code):
    assert _rope(**kw) == code


@pytest.mark.parametrize("kw,code", [
    # more heads than a launch has threads for, and products of sizes beyond 64 bits
    (dict(T=1 << 23), EUNSUP), (dict(T=1 << 62, Hq=0, Hkv=2), EUNSUP), (dict(T=1 << 61), EUNSUP),
    (dict(pages=1 << 40, page=1 << 30, ps=128 << 30), EUNSUP),
    (dict(pages=4, page=2, hs=1 << 62, ts=64, ps=1 << 62), EINVAL),  # the second page on the second head
])
def test_rope_refuses_sizes_beyond_a_launch(kw, code):
    assert _rope(**kw) == code


def _attn(**kw):
    a = dict(dtype=1, T=4, G=2, Hq=4, Hkv=2, D=64, pages=8, page=16, q=0x1000, ldq=256, kc=0x2000, vc=0x3000,
             ps=16 * 128, ts=128, hs=64, indptr=0x4000, perm=None, pp=0x5000, wp=4, pl=0x6000, op=0x7000, wo=4,
             ol=0x8000, scale=0.125, out=0x9000, ldo=256, lse=None, ws=0x10000, nbytes=1 << 40, stream=None)
    a.update(kw)
    return _lib.lib().lora_prefix_attention(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), EUNSUP), (dict(T=-1), EINVAL), (dict(G=-1), EINVAL), (dict(Hq=0), EINVAL), (dict(Hkv=0), EINVAL),
    (dict(Hq=5), EINVAL), (dict(D=0), EINVAL), (dict(D=60), EUNSUP), (dict(D=264), EUNSUP), (dict(pages=-1), EINVAL),
    (dict(pages=1 << 31), EUNSUP), (dict(page=0), EINVAL), (dict(wp=-1), EINVAL), (dict(wo=-1), EINVAL),
    (dict(wp=1 << 27), EUNSUP), (dict(wo=1 << 27), EUNSUP), (dict(T=1 << 25), EUNSUP),
    (dict(T=1 << 24, Hq=8, ldq=512, ldo=512), EUNSUP), (dict(scale=nan), EINVAL), (dict(scale=inf), EINVAL),
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(indptr=None), EINVAL), (dict(pp=None), EINVAL),
    (dict(pl=None), EINVAL), (dict(op=None), EINVAL), (dict(ol=None), EINVAL), (dict(kc=None), EINVAL),
    (dict(vc=None), EINVAL), (dict(ldq=255), EINVAL), (dict(ldo=255), EINVAL), (dict(ldq=260), EUNSUP),
    (dict(q=0x1002), EUNSUP), (dict(kc=0x2008), EUNSUP), (dict(vc=0x3008), EUNSUP), (dict(ps=-8), EINVAL),
    (dict(ps=2052), EUNSUP), (dict(ts=132), EUNSUP), (dict(hs=68), EUNSUP), (dict(ws=None), EWS),
    (dict(nbytes=100), EWS), (dict(ws=0x10008), EWS), (dict(T=0, q=None, out=None, ws=None), OK),
    (dict(G=0, q=None, ws=None), OK),
])
def test_attention_refusals(kw, code):
    assert _attn(**kw) == code


@pytest.mark.parametrize("kw", [
    dict(T=1 << 24, Hq=4, Hkv=1),             # one thread too many in the join
    dict(T=1 << 23, Hq=4, Hkv=4, ldq=256),    # a workgroup per token and key head, of 256 threads
])
def test_attention_refuses_batches_beyond_a_launch(kw):
    assert _attn(wp=0, nbytes=1 << 60, **kw) == EUNSUP


def test_attention_workspace_query():
    size = _lib.lora_prefix_attention_workspace_size
    assert size(1, 4, 2, 4, 2, 64, 16, 4, 4) > 0
    for bad in ((0, 4, 2, 4, 2, 64, 16, 4, 4), (1, 4, 2, 5, 2, 64, 16, 4, 4), (1, 0, 2, 4, 2, 64, 16, 4, 4),
                (1, 4, 0, 4, 2, 64, 16, 4, 4), (1, 4, 2, 4, 2, 60, 16, 4, 4), (1, 4, 2, 4, 2, 64, 16, 0, 0)):
        assert size(*bad) == 0


# ------------------------------------------------------------------------------- the tensor wrappers

@pytest.fixture
def no_device_check(monkeypatch):
    monkeypatch.setattr(ops, "_dev", lambda *ts: None)


def _refused(call, kinds=(ValueError, TypeError)):
    """The call is refused for its own fault: the check of the device is the last one, so CPU tensors
    stand in for device ones."""
    with pytest.raises(kinds) as e:
        call()
    assert "GPU" not in str(e.value), e.value


def test_cpu_tensors_are_refused():
    z = torch.zeros(4, 64, dtype=bf)
    with pytest.raises(ValueError, match="GPU"):
        d.linear_w4_prepare(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=bf))
    with pytest.raises(ValueError, match="GPU"):
        d.linear_w4(z, d.W4Weight(torch.zeros(2304, dtype=torch.uint8), bf, 64, 4, 64, False))
    with pytest.raises(ValueError, match="GPU"):
        d.rope_append(**_rope_tensors())
    with pytest.raises(ValueError, match="GPU"):
        d.prefix_attention(**_attn_tensors())


@pytest.mark.parametrize("codes,scales,zp", [
    (torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 1, dtype=bf), None),
    (torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(5, 1, dtype=bf), None),
    (torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 3, dtype=bf), None),
    (torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 0, dtype=bf), None),
    (torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 4, dtype=bf), None),   # group 16
    (torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1), None),             # float32 scales
    (torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=bf), torch.zeros(4, 2, dtype=torch.uint8)),
    (torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=bf), torch.zeros(4, 1, dtype=torch.int32)),
    (torch.zeros(32, 4, dtype=torch.uint8).t(), torch.zeros(4, 1, dtype=bf), None),
])
def test_w4_prepare_wrapper(no_device_check, codes, scales, zp):
    with pytest.raises((ValueError, TypeError)):
        d.linear_w4_prepare(codes, scales, zp)


def test_w4_wrapper():
    w = d.W4Weight(torch.zeros(2304, dtype=torch.uint8), bf, 64, 4, 64, False)
    _refused(lambda: d.linear_w4(torch.zeros(2, 64, dtype=bf), d.W4Weight(w.data[:1024], bf, 64, 4, 64, False)))
    for x, out in ((torch.zeros(2, 64), None), (torch.zeros(2, 32, dtype=bf), None),
                   (torch.zeros(64, 2, dtype=bf).t(), None), (torch.zeros(2, 64, dtype=bf), torch.zeros(2, 5, dtype=bf)),
                   (torch.zeros(2, 64, dtype=bf), torch.zeros(2, 4))):
        _refused(lambda: d.linear_w4(x, w, out))
    w = d.W4Weight(torch.zeros(2304, dtype=torch.uint8), bf, 64, 4, 64, False)
    with pytest.raises(ValueError, match="GPU"):  # sizes right, nothing left but the device
        d.linear_w4(torch.zeros(2, 64, dtype=bf), w)


def _rope_tensors(**kw):
    a = dict(q=torch.zeros(3, 128, dtype=bf), k=torch.zeros(3, 64, dtype=bf), v=torch.zeros(3, 64, dtype=bf),
             table=torch.zeros(10, 64), positions=torch.zeros(3, dtype=torch.int32),
             slots=torch.zeros(3, dtype=torch.int64), k_cache=torch.zeros(2, 4, 1, 64, dtype=bf),
             v_cache=torch.zeros(2, 4, 1, 64, dtype=bf))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 100, dtype=bf)), dict(q=torch.zeros(128, 3, dtype=bf).t()), dict(k=torch.zeros(3, 64)),
    dict(k=torch.zeros(2, 64, dtype=bf)), dict(v=torch.zeros(3, 32, dtype=bf)), dict(table=torch.zeros(10, 64, dtype=bf)),
    dict(table=torch.zeros(64, 10).t()), dict(positions=torch.zeros(3, dtype=torch.int64)),
    dict(positions=torch.zeros(2, dtype=torch.int32)), dict(slots=torch.zeros(3, dtype=torch.int32)),
    dict(slots=torch.zeros(4, dtype=torch.int64)), dict(k_cache=torch.zeros(2, 4, 1, 64)),
    dict(v_cache=torch.zeros(2, 5, 1, 64, dtype=bf)), dict(v_cache=torch.zeros(4, 2, 1, 64, dtype=bf).transpose(0, 1)),
    dict(k_cache=torch.zeros(2, 64, 1, 4, dtype=bf).transpose(1, 3), v_cache=torch.zeros(2, 64, 1, 4, dtype=bf).transpose(1, 3)),
    dict(q_norm=torch.zeros(63, dtype=bf)), dict(k_norm=torch.zeros(64)), dict(q_out=torch.zeros(3, 64, dtype=bf)),
    dict(q_out=torch.zeros(3, 128)),
])
def test_rope_wrapper(kw):
    _refused(lambda: d.rope_append(**_rope_tensors(**kw)))


def _attn_tensors(**kw):
    i = torch.int32
    a = dict(q=torch.zeros(3, 128, dtype=bf), k_cache=torch.zeros(2, 4, 1, 64, dtype=bf),
             v_cache=torch.zeros(2, 4, 1, 64, dtype=bf), seg_indptr=torch.tensor([0, 3], dtype=i),
             permutation=torch.arange(3, dtype=i), prefix_pages=torch.zeros(1, 2, dtype=i),
             prefix_lens=torch.zeros(1, dtype=i), own_pages=torch.zeros(3, 2, dtype=i),
             own_lens=torch.zeros(3, dtype=i), scale=0.125)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 128)), dict(q=torch.zeros(3, 100, dtype=bf)), dict(k_cache=torch.zeros(2, 4, 1, 64)),
    dict(seg_indptr=torch.zeros(2, dtype=torch.int64)), dict(seg_indptr=torch.zeros(0, dtype=torch.int32)),
    dict(permutation=torch.zeros(2, dtype=torch.int32)), dict(prefix_pages=torch.zeros(2, 2, dtype=torch.int32)),
    dict(prefix_pages=torch.zeros(1, 2, dtype=torch.int64)), dict(prefix_pages=None), dict(prefix_lens=None),
    dict(prefix_lens=torch.zeros(2, dtype=torch.int32)), dict(own_pages=torch.zeros(2, 2, dtype=torch.int32)),
    dict(own_pages=torch.zeros(2, 3, dtype=torch.int32).t()), dict(own_lens=None), dict(out=torch.zeros(3, 64, dtype=bf)),
    dict(out=torch.zeros(3, 128)), dict(workspace=torch.zeros(4)),
])
def test_attention_wrapper(kw):
    _refused(lambda: d.prefix_attention(**_attn_tensors(**kw)))


def test_outputs_must_not_overlap_inputs():
    buf = torch.zeros(4 * 256, dtype=bf)
    w = d.W4Weight(torch.zeros(4 * 1024 + 256, dtype=torch.uint8), bf, 64, 64, 64, False)
    x = buf[:256].view(4, 64)
    wide = buf.view(4, 256)
    for out in (x, buf[64:320].view(4, 64), wide[:, 32:96]):
        _refused(lambda: d.linear_w4(x, w, out))
    _refused(lambda: d.linear_w4(wide[:, :64], w, wide[:, 40:104]))
    for xx, out in ((wide[:, :64], wide[:, 64:128]), (wide[:, 192:], wide[:, :64]), (x, buf[256:512].view(4, 64))):
        with pytest.raises(ValueError, match="GPU"):  # nothing left but the device
            d.linear_w4(xx, w, out)
    q = torch.zeros(4, 128, dtype=bf)
    _refused(lambda: d.prefix_attention(**_attn_tensors(q=q[:3], out=q[:3])))
    _refused(lambda: d.prefix_attention(**_attn_tensors(q=q[:3], out=q[1:])))
    _refused(lambda: d.rope_append(**_rope_tensors(q=q[:3], q_out=q[1:])))
    with pytest.raises(ValueError, match="GPU"):
        d.rope_append(**_rope_tensors(q=q[:3], q_out=q[:3]))


@pytest.mark.parametrize("kw", [dict(q="x"), dict(k_cache=None), dict(scale="x"), dict(own_pages=3)])
def test_attention_wrapper_types(kw):
    _refused(lambda: d.prefix_attention(**_attn_tensors(**kw)), TypeError)


def test_status_becomes_an_error():
    with pytest.raises(_lib.LoraError, match="WORKSPACE"):
        d._result("lora_prefix_attention", EWS)
