"""GPU parity of the decode-step operators (linear_w4, rope_append, prefix_attention) against the
fp64 oracle, at the sizes, masks, strides and orders where they can go wrong, and a run of them
together with the multi-adapter update. Tolerances: tests/decode_cases.py."""

import numpy as np
import pytest
import torch

import oracle
from tests import decode_cases as dc
from tests.decode_cases import DT, f64, within

pytestmark = pytest.mark.gpu

lm = __import__("adapter_lora_projection_amd")
dev = lambda t: None if t is None else t.to("cuda")


# ---------------------------------------------------------------------------------- linear_w4

def _w4(x, codes, scales, zp, **kw):
    w = lm.linear_w4_prepare(dev(codes), dev(scales), dev(zp))
    return lm.linear_w4(x if x.is_cuda else dev(x), w, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,group,zeros", [
    (1, 32, 1, 32, False), (1, 96, 17, 32, True), (3, 128, 16, 128, True), (16, 192, 33, 64, False),
    (17, 1056, 1000, 32, True), (33, 640, 70, 128, False), (70, 256, 48, 64, True),
    (1, 4096, 512, 128, False), (2, 16384, 64, 64, True), (130, 128, 130, 32, True),
    (8, 4096, 4096, 128, True), (64, 2048, 272, 128, True),
    # ranges of K in fp32 planes (16, 32 and 64 rows a workgroup), and slabs over all of K
    (16, 16384, 72, 128, False), (24, 8192, 260, 64, True), (24, 8192, 260, 32, True), (33, 12288, 100, 128, True),
    (40, 256, 16500, 64, False), (64, 128, 20000, 128, True), (20, 96, 30000, 32, True), (5, 32, 50000, 32, False),
])
def test_w4(dtype, M, K, N, group, zeros):
    print("w4", dtype, M, K, N, group, zeros, flush=True)
    x, codes, scales, zp = dc.w4_inputs(M * 7 + K + N, dtype, M, K, N, group, zeros)
    y = _w4(x, codes, scales, zp)
    ref = oracle.linear_w4(x, codes, scales, zp)
    within(f64(y), ref, dc.w4_bound(dtype, x, scales, ref, group), "y")
    again = _w4(x, codes, scales, zp)
    assert torch.equal(y, again)


@pytest.mark.parametrize("M,K", [(6, 160), (33, 160), (40, 12320)])
def test_w4_strided_rows_and_output(M, K):
    x, codes, scales, zp = dc.w4_inputs(5, "bf16", M, K, 37, 32, True)
    wide = torch.full((M, K + 40), float("nan"), dtype=DT["bf16"])
    wide[:, :K] = x
    out = torch.full((M, 51), 7.0, dtype=DT["bf16"], device="cuda")
    pad = torch.cat([codes, codes[:, :8]], 1)  # strided codes, scales and zero points too
    sc, z = torch.cat([scales, scales], 1), torch.cat([zp, zp], 1)
    w = lm.linear_w4_prepare(dev(pad)[:, :K // 2], dev(sc)[:, :K // 32], dev(z)[:, :K // 32])
    lm.linear_w4(dev(wide)[:, :K], w, out=out[:, 3:40])
    ref = oracle.linear_w4(x, codes, scales, zp)
    within(f64(out[:, 3:40]), ref, dc.w4_bound("bf16", x, scales, ref, 32), "y")
    assert torch.all(out[:, :3] == 7.0) and torch.all(out[:, 40:] == 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", [256, 16384])
def test_w4_rows_do_not_mix(dtype, K):
    """A NaN row of x gives a NaN row of y and leaves the others as they were; a NaN scale its own
    column."""
    x, codes, scales, zp = dc.w4_inputs(9, dtype, 21, K, 40, 128, True)
    y0 = _w4(x, codes, scales, zp)
    x[20] = float("nan")
    scales[7, 1] = float("nan")
    y1 = _w4(x, codes, scales, zp)
    assert torch.isnan(y1[20]).all() and torch.isnan(y1[:, 7]).all()
    keep = [c for c in range(40) if c != 7]
    assert torch.equal(y0[:20, keep], y1[:20, keep])


def test_w4_no_rows_writes_nothing():
    _, codes, scales, _ = dc.w4_inputs(3, "bf16", 1, 64, 32, 32, False)
    w = lm.linear_w4_prepare(dev(codes), dev(scales))
    assert lm.linear_w4(torch.empty((0, 64), dtype=DT["bf16"], device="cuda"), w).shape == (0, 32)


def test_w4_large_scale_range():
    """Scales far apart in one row: every group's offset leaves before the groups are added."""
    x, codes, scales, zp = dc.w4_inputs(11, "bf16", 4, 512, 32, 128, True)
    scales[:, 0] *= 1024
    scales[:, 2] /= 1024
    ref = oracle.linear_w4(x, codes, scales, zp)
    within(f64(_w4(x, codes, scales, zp)), ref, dc.w4_bound("bf16", x, scales, ref, 128), "y")


# ---------------------------------------------------------------------------------- rope_append

def _rope_case(seed, dtype, T, Hq, Hkv, D, rot, page, norm, layout="phd", rows=40, gap=0):
    g = dc.gen(seed)
    qkv = dc.normal(g, (T, (Hq + 2 * Hkv) * D + gap), dtype)
    pages = (2 * T + page - 1) // page + 1
    shape = (pages, page, Hkv, D) if layout == "phd" else (pages, Hkv, page, D)
    kc, vc = dc.normal(g, shape, dtype), dc.normal(g, shape, dtype)
    pos = torch.randint(0, rows, (T,), generator=g, dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:T]
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(DT[dtype]) if norm else None for _ in range(2)]
    return qkv, kc, vc, pos, slots, w


def _views(qkv, Hq, Hkv, D):
    return qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D]


def _check_rope(got_q, got_k, got_v, ref, dtype, D, rot, inter):
    q, k, v = ref
    qh = q.reshape(q.shape[0], -1, D)
    within(f64(got_q).reshape(qh.shape), qh, dc.rope_bound(dtype, qh, D, rot, inter), "q")
    within(f64(got_k), k, dc.rope_bound(dtype, k, D, rot, inter), "k cache")
    assert np.array_equal(f64(got_v), v)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,inter,norm,layout,gap", [
    (1, 1, 1, 2, 2, 1, False, False, "phd", 0),
    (5, 4, 2, 64, 64, 16, False, True, "phd", 0),
    (7, 6, 3, 80, 32, 5, True, True, "hpd", 8),
    (9, 2, 2, 128, 64, 16, False, True, "hpd", 0),
    (300, 8, 1, 128, 128, 64, False, True, "phd", 16),
    (4, 3, 1, 256, 256, 7, True, False, "phd", 0),
    (3, 2, 1, 256, 128, 24, False, True, "phd", 0),
    (6, 3, 2, 20, 6, 3, False, True, "phd", 1),     # odd sizes: the element form
    (6, 3, 2, 21, 10, 3, True, True, "hpd", 3),
    (2, 2, 1, 130, 128, 3, False, True, "phd", 0),
    (3, 2, 1, 72, 16, 4, False, True, "phd", 0),    # an odd number of 8-element chunks
    (2, 1, 1, 1024, 1024, 2, False, True, "phd", 0),
    (3, 0, 2, 64, 64, 4, False, False, "phd", 0),   # keys and values alone
])
def test_rope_append(dtype, T, Hq, Hkv, D, rot, page, inter, norm, layout, gap):
    print("rope", dtype, T, Hq, Hkv, D, rot, page, inter, norm, layout, gap, flush=True)
    qkv, kc, vc, pos, slots, (wq, wk) = _rope_case(T + D, dtype, T, Hq, Hkv, D, rot, page, norm, layout, gap=gap)
    tab = dc.table(40, rot)
    if layout == "hpd":
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    q, k, v = _views(qkv, Hq, Hkv, D)
    ref = oracle.rope_append(q, k, v, tab, pos, slots, kc, vc, wq, wk, 1e-6, inter)
    d = dev(qkv)
    qd, kd, vd = _views(d, Hq, Hkv, D)
    kcd, vcd = dev(kc), dev(vc)
    assert kcd.stride() == kc.stride()
    got = lm.rope_append(qd, kd, vd, dev(tab), dev(pos), dev(slots), kcd, vcd, dev(wq), dev(wk), 1e-6, inter)
    _check_rope(got, kcd, vcd, ref, dtype, D, rot, inter)
    assert torch.equal(d.cpu(), qkv)  # inputs unchanged
    if Hq:
        lm.rope_append(qd, kd, vd, dev(tab), dev(pos), dev(slots), kcd, vcd, dev(wq), dev(wk), 1e-6, inter,
                       q_out=qd)
        assert torch.equal(qd.contiguous(), got)  # in place, the same values


@pytest.mark.parametrize("D,rot", [(64, 64), (20, 6)])
def test_rope_rows_left_out(D, rot):
    """Positions outside the table leave a token out, slots outside the cache append nothing, and
    nothing else of the cache or of q_out changes."""
    T, Hq, Hkv, page = 8, 2, 2, 4
    qkv, kc, vc, pos, slots, _ = _rope_case(3, "bf16", T, Hq, Hkv, D, rot, page, False)
    n = kc.shape[0] * page
    pos[1], pos[2] = -1, 40
    slots[3], slots[4], slots[5], slots[6] = -1, n, 2 ** 40, -2 ** 62
    tab = dc.table(40, rot)
    q, k, v = _views(qkv, Hq, Hkv, D)
    ref = oracle.rope_append(q, k, v, tab, pos, slots, kc, vc)
    d, kcd, vcd = dev(qkv), dev(kc), dev(vc)
    out = torch.full((T, Hq * D), float("nan"), dtype=DT["bf16"], device="cuda")
    lm.rope_append(*_views(d, Hq, Hkv, D), dev(tab), dev(pos), dev(slots), kcd, vcd, q_out=out)
    _check_rope(out, kcd, vcd, ref, "bf16", D, rot, False)
    assert torch.isnan(out[1:3]).all() and not torch.isnan(out[3:]).any()


def test_rope_copies_v_bits():
    """v is copied, not converted: signalling NaNs and both zeros keep their bits."""
    T, H, D = 4, 1, 64
    bits = torch.arange(T * H * D, dtype=torch.int32) * 257 + 0x7f00
    for dt in (torch.bfloat16, torch.float16):
        v = (bits & 0xffff).to(torch.int32).sub((bits & 0x8000) * 2).to(torch.int16).view(dt).view(T, H * D)
        q = torch.zeros((T, H * D), dtype=dt)
        kc = torch.zeros((T, 1, H, D), dtype=dt, device="cuda")
        vc = torch.zeros_like(kc)
        lm.rope_append(dev(q), dev(q), dev(v), dev(dc.table(4, D)), dev(torch.arange(T, dtype=torch.int32)),
                       dev(torch.arange(T)), kc, vc)
        assert torch.equal(vc.view(torch.int16).cpu().view(T, -1), v.view(torch.int16))


# ---------------------------------------------------------------------------------- prefix_attention

ATTN = {
    # name: (T, segment lengths, Hq, Hkv, D, page, prefix lengths, own lengths, options)
    "one token, one key": (1, [1], 1, 1, 8, 1, [0], [1], {}),
    "one prefix key": (2, [2], 2, 1, 64, 16, [1], [0, 0], {}),
    "empty everywhere": (3, [2, 1], 4, 2, 64, 4, [0, 0], [0, 0, 0], {}),
    "some rows empty": (5, [2, 3], 4, 2, 128, 4, [0, 9], [0, 3, 0, 1, 0], {}),
    "negative lengths": (3, [3], 2, 2, 64, 4, [-5], [7, -1, 2], {}),
    "empty segments": (6, [0, 4, 0, 0, 2], 4, 4, 64, 16, [3, 40, 0, 17, 64], [1, 2, 3, 4, 5, 6], {}),
    "uncovered rows": (9, [3, 2], 4, 2, 64, 8, [33, 5], [9] * 9, dict(indptr0=2)),
    "odd head": (4, [4], 7, 1, 72, 5, [101], [3, 50, 31, 32], {}),
    "d80": (7, [3, 4], 28, 4, 80, 24, [199, 100], [1, 23, 24, 25, 48, 49, 70], {}),
    "block edges": (8, [8], 4, 1, 128, 16, [128], [31, 32, 33, 63, 64, 65, 127, 129], {}),
    "d256": (5, [2, 3], 4, 2, 256, 16, [300, 257], [5, 64, 65, 200, 1], {}),
    "d248": (3, [3], 2, 1, 248, 3, [70], [5, 6, 64], {}),
    "16 to 1": (5, [5], 16, 1, 64, 32, [100], [10, 20, 30, 40, 50], {}),
    "40 to 1": (3, [3], 40, 1, 64, 32, [70], [10, 20, 300], {}),
    "heads before places": (6, [4, 2], 8, 4, 128, 16, [90, 33], [3, 17, 40, 1, 0, 5], dict(layout="hpd")),
    "identity order": (6, [4, 2], 8, 4, 64, 16, [90, 33], [3, 17, 40, 1, 0, 5], dict(perm=False)),
    "strided q": (6, [6], 8, 4, 64, 16, [50], [3, 17, 40, 1, 0, 5], dict(q_pad=24)),
    "many segments": (70, [1] * 70, 2, 1, 64, 4, list(range(70)), [(7 * t) % 11 for t in range(70)], {}),
    "long": (3, [2, 1], 4, 2, 128, 64, [5000, 4097], [1200, 3, 2049], {}),
    "many rows": (150, [100, 50], 8, 2, 64, 16, [700, 333], [(13 * t) % 70 for t in range(150)], {}),
    "many rows d128": (90, [70, 20], 8, 2, 128, 16, [1500, 640], [(29 * t) % 90 for t in range(90)], {}),
    "many rows d256": (40, [33, 7], 8, 1, 256, 16, [500, 64], [(29 * t) % 90 for t in range(40)], {}),
    "pages of one place": (9, [9], 8, 2, 128, 1, [300], [(29 * t) % 90 for t in range(9)], {}),
    "one page each": (20, [20], 8, 2, 64, 1000, [900], [(29 * t) % 90 for t in range(20)], {}),
    "sharp": (12, [12], 8, 2, 128, 16, [900], [(29 * t) % 90 for t in range(12)], dict(std=6.0)),
}


def _attn(c, **kw):
    return lm.prefix_attention(*c.args(dev), return_lse=True, **kw)


def _check_attn(c, out, lse, what="out"):
    ref, rl, spread = oracle.prefix_attention(*c.args())
    bo, bl = c.bounds(ref, rl, spread)
    cov = ~np.isnan(rl[:, 0])
    within(f64(out)[cov], ref[cov], bo[cov], what)
    within(f64(lse)[cov], rl[cov], bl[cov], what + " lse")
    return cov


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", list(ATTN))
def test_attention(dtype, name):
    print("attention", dtype, name, flush=True)
    T, segs, Hq, Hkv, D, page, pre, own, opt = ATTN[name]
    c = dc.Attn(len(name) * 31 + T, dtype, T, segs, Hq, Hkv, D, page, pre, own, **opt)
    mark = torch.full((T, Hq * D), 7.0, dtype=DT[dtype], device="cuda")
    out, lse = _attn(c, out=mark)
    cov = _check_attn(c, out, lse)
    assert torch.all(out[torch.from_numpy(~cov).cuda()] == 7.0)  # rows no segment covers
    out2, lse2 = _attn(c)
    rows = torch.from_numpy(cov).cuda()
    assert torch.equal(out2[rows], out[rows]) and torch.equal(lse2[rows], lse[rows])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_pages_outside_the_cache_are_masked(D):
    c = dc.Attn(5, "bf16", 40, [33, 7], 8, 2, D, 16, [150, 40], [20] * 40)
    c.prefix_pages[0, 2], c.prefix_pages[0, 9] = -1, c.k.shape[0]
    c.prefix_pages[1, :] = 2 ** 31 - 1  # all of the second prefix
    c.own_pages[3, 0], c.own_pages[4, 1], c.own_pages[5, :] = -2 ** 31, 2 ** 30, -7
    _check_attn(c, *_attn(c))


def test_attention_lengths_beyond_the_lists_are_clamped():
    c = dc.Attn(6, "f16", 3, [3], 4, 2, 64, 16, [32], [16, 16, 16], extra_pages=0)
    c.prefix_lens[0] = 2 ** 31 - 1
    c.own_lens[1] = 100
    _check_attn(c, *_attn(c))


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30])
@pytest.mark.parametrize("T", [3, 40])
def test_attention_other_scales(scale, T):
    """Equal weights, a negative scale, a tiny one: masked places stay out of all of them."""
    c = dc.Attn(7, "bf16", T, [T], 8, 2, 128, 16, [100], [(7 * t) % 33 for t in range(T)])
    c.scale = scale
    ref, rl, spread = oracle.prefix_attention(*c.args())
    bo, bl = c.bounds(ref, rl, spread)
    c.scale = abs(scale)
    bo2, bl2 = c.bounds(ref, rl, spread)  # the bound takes the magnitude
    c.scale = scale
    out, lse = _attn(c)
    within(f64(out), ref, np.maximum(bo, bo2), "out")
    within(f64(lse), rl, np.maximum(bl, bl2), "lse")


def test_empty_batches():
    z = lambda *s, d="bf16": torch.zeros(s, dtype=DT.get(d, d), device="cuda")
    kc = z(2, 4, 2, 64)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    q = lm.rope_append(z(0, 256), z(0, 128), z(0, 128), dev(dc.table(4, 64)), i32(0),
                       torch.zeros(0, dtype=torch.int64, device="cuda"), kc, kc.clone())
    assert q.shape == (0, 256)
    out, lse = lm.prefix_attention(q, kc, kc, i32(3), None, i32(2, 1), i32(2), i32(0, 1), i32(0), 0.1, return_lse=True)
    assert out.shape == (0, 256) and lse.shape == (0, 4)
    mark = torch.full((3, 256), 7.0, dtype=DT["bf16"], device="cuda")  # no segment: nothing is written
    lm.prefix_attention(z(3, 256), kc, kc, i32(1), None, i32(0, 1), i32(0), i32(3, 1), i32(3), 0.1, out=mark)
    # a cache without pages: every key is masked, every row empty
    out = lm.prefix_attention(z(3, 256), kc[:0], kc[:0], dev(torch.tensor([0, 3], dtype=torch.int32)), None, i32(1, 2),
                              i32(1) + 5, i32(3, 2), i32(3) + 4, 0.1)
    assert torch.all(mark == 7.0) and torch.all(out == 0)


def test_attention_without_prefixes_or_own_keys():
    c = dc.Attn(8, "bf16", 5, [3, 2], 4, 2, 64, 16, [40, 70], [5, 6, 7, 30, 0])
    both = f64(_attn(c)[0])
    for drop in ("prefix", "own", "both"):
        d = dc.Attn(8, "bf16", 5, [3, 2], 4, 2, 64, 16, [40, 70], [5, 6, 7, 30, 0])
        if drop in ("prefix", "both"):
            d.prefix_lens[:] = 0
        if drop in ("own", "both"):
            d.own_lens[:] = 0
        a = list(d.args(dev))
        if drop in ("prefix", "both"):
            a[5] = a[6] = None
        if drop in ("own", "both"):
            a[7] = a[8] = None
        out, lse = lm.prefix_attention(*a, return_lse=True)
        _check_attn(d, out, lse, drop)
        assert drop == "both" or not np.array_equal(f64(out), both)


def test_refusals_of_the_library_on_the_gpu():
    """What only the library can refuse raises before anything is written."""
    c = dc.Attn(8, "bf16", 5, [3, 2], 4, 2, 64, 16, [40, 70], [5, 6, 7, 30, 0])
    out = torch.full((5, 256), 7.0, dtype=DT["bf16"], device="cuda")
    err = lm.LoraError
    with pytest.raises(err, match="WORKSPACE"):
        lm.prefix_attention(*c.args(dev), out=out, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    a = list(c.args(dev))
    with pytest.raises(err, match="UNSUPPORTED"):  # rows of q off the 16-byte grid
        lm.prefix_attention(torch.zeros((5, 260), dtype=DT["bf16"], device="cuda")[:, 2:258], *a[1:], out=out)
    with pytest.raises(err, match="EINVAL"):
        lm.prefix_attention(*a[:9], float("nan"), out=out)
    with pytest.raises(ValueError, match="GPU"):
        lm.prefix_attention(c.q, *a[1:], out=out)
    k = a[1].expand(a[1].shape)
    with pytest.raises(err, match="EINVAL"):  # places that overlap
        lm.rope_append(a[0], a[0][:, :128], a[0][:, :128], dev(dc.table(4, 64)), dev(torch.zeros(5, dtype=torch.int32)),
                       dev(torch.arange(5)), k[:1].expand(4, -1, -1, -1), k[:1].expand(4, -1, -1, -1))
    w = lm.linear_w4_prepare(torch.zeros((16, 32), dtype=torch.uint8, device="cuda"), torch.ones((16, 1), dtype=DT["f16"], device="cuda"))
    with pytest.raises(err, match="UNSUPPORTED"):
        lm.linear_w4(torch.zeros((2, 66), dtype=DT["f16"], device="cuda")[:, 1:65], w)
    torch.cuda.synchronize()
    assert torch.all(out == 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,page,first,layout", [
    (70, 16, 8, 128, 16, 0, "phd"), (70, 8, 8, 64, 3, 2, "hpd"), (40, 40, 20, 80, 24, 1, "phd"),
    (80, 80, 8, 256, 16, 0, "phd"), (600, 20, 1, 64, 32, 0, "phd"),
])
def test_attention_one_range_per_row(dtype, T, Hq, Hkv, D, page, first, layout):
    """Enough rows for one key range each and no prefix: written without a join. Rows without keys,
    rows without a segment, output rows off the 8-byte grid, pages outside the cache."""
    own = [(17 * t) % 70 for t in range(T)]
    own[T // 2] = 0
    c = dc.Attn(T + D, dtype, T, [T // 2, T - first - T // 2 - 1], Hq, Hkv, D, page, [0, 0], own, indptr0=first, layout=layout)
    c.own_pages[5, 0] = -1
    a = list(c.args(dev))
    a[5] = a[6] = None
    mark = torch.full((T, Hq * D + 3), 7.0, dtype=DT[dtype], device="cuda")
    assert lm.prefix_attention_workspace(a[0], a[1], a[3], None, a[7]).numel() == 0
    out, lse = lm.prefix_attention(*a, return_lse=True, out=mark[:, 1:1 + Hq * D])
    cov = _check_attn(c, out, lse)
    assert cov.sum() == T - first - 1 and torch.all(out[torch.from_numpy(~cov).cuda()] == 7.0)
    assert torch.all(mark[:, 0] == 7.0) and torch.all(mark[:, 1 + Hq * D:] == 7.0)
    aligned = lm.prefix_attention(*a)
    assert torch.equal(aligned[torch.from_numpy(cov).cuda()], out[torch.from_numpy(cov).cuda()])


@pytest.mark.parametrize("T,Hq,Hkv", [(3, 4, 2), (9, 16, 1), (70, 8, 1)])
def test_attention_many_empty_segments(T, Hq, Hkv):
    """More segments than rows, and rows in the first, a middle and the last of them."""
    lens = [0] * 300
    lens[0], lens[150], lens[299] = 1, T - 2, 1
    c = dc.Attn(T, "bf16", T, lens, Hq, Hkv, 64, 16, [(7 * g) % 90 for g in range(300)], [5] * T)
    print("segments", T, Hq, Hkv, flush=True)
    out, lse = lm.prefix_attention(*c.args(dev), return_lse=True)
    assert _check_attn(c, out, lse).all()


def test_attention_same_sequence_several_tokens():
    """Tokens of one sequence as rows that repeat its pages with lengths rising by one."""
    c = dc.Attn(9, "bf16", 6, [6], 8, 2, 128, 16, [100], [37] * 6)
    c.own_pages[1:] = c.own_pages[0]
    c.own_lens[:] = torch.arange(32, 38, dtype=torch.int32)
    _check_attn(c, *_attn(c))


def test_attention_offsets_beyond_32_bits():
    """Pages whose elements lie past 2^31 (and byte offsets past 2^32)."""
    page, Hkv, D = 64, 8, 128
    pages = (1 << 31) // (page * Hkv * D) + 40
    c = dc.Attn(10, "bf16", 4, [4], 16, Hkv, D, page, [200], [70, 3, 64, 65])
    n = c.k.shape[0]
    big = [torch.empty((pages, page, Hkv, D), dtype=DT["bf16"], device="cuda") for _ in range(2)]
    big[0][pages - n:], big[1][pages - n:] = dev(c.k), dev(c.v)
    a = list(c.args(dev))
    a[1], a[2], a[5], a[7] = big[0], big[1], a[5] + (pages - n), a[7] + (pages - n)
    out, lse = lm.prefix_attention(*a, return_lse=True)
    _check_attn(c, out, lse)
    # and the append into the same places
    kv = dc.normal(dc.gen(1), (1, Hkv * D), "bf16")
    slot = torch.tensor([pages * page - 1])
    lm.rope_append(dev(kv), dev(kv), dev(kv), dev(dc.table(2, D)), dev(torch.zeros(1, dtype=torch.int32)),
                   dev(slot), *big)
    assert torch.equal(big[1][-1, -1].cpu().view(1, -1), kv)
    assert torch.equal(big[0][-1, -1].cpu().view(1, -1), kv)  # position 0: cos 1, sin 0


# ---------------------------------------------------------------------------------- together

class Step:
    """One decode step of an attention layer under several adapters on a 4-bit base, in the order a
    server makes the calls."""

    T, H, Hq, Hkv, D, page, R = 12, 256, 4, 2, 64, 16, 16

    def __init__(self, seed):
        g = dc.gen(seed)
        H, Hq, Hkv, D, T = self.H, self.Hq, self.Hkv, self.D, self.T
        N = (Hq + 2 * Hkv) * D
        self.c = dc.Attn(seed, "bf16", T, [5, 3, 4], Hq, Hkv, D, self.page, [70, 33, 0],
                         [1 + (5 * t) % 40 for t in range(T)])
        self.x = dc.normal(g, (T, H), "bf16")
        _, self.wqkv, self.sqkv, self.zqkv = dc.w4_inputs(seed + 1, "bf16", 1, H, N, 64, True)
        _, self.wo, self.so, self.zo = dc.w4_inputs(seed + 2, "bf16", 1, Hq * D, H, 128, False)
        L, R = 3, self.R
        self.A = dc.normal(g, (L, 3 * R, H), "bf16", 0.05)
        self.B = dc.normal(g, (L, N, R), "bf16", 0.1)
        self.Ao = dc.normal(g, (L, R, Hq * D), "bf16", 0.05)
        self.Bo = dc.normal(g, (L, H, R), "bf16", 0.1)
        i32 = lambda a: torch.tensor(a, dtype=torch.int32)
        self.meta = dict(indptr=self.c.indptr, widx=i32([2, 0, 1]), perm=self.c.perm, ranks=i32([16, 8, 3]),
                         off=i32([0, Hq * D, (Hq + Hkv) * D, N]), off_o=i32([0, H]), sc=torch.tensor([0.5, 2.0, 1.0]))
        self.table = dc.table(300, D)
        self.qn = (1 + 0.2 * torch.randn(D, generator=g)).to(DT["bf16"])
        # the new key goes to the last own place; its position is prefix + own length - 1
        seg_of = np.repeat(np.arange(3), [5, 3, 4])
        pre = self.c.prefix_lens.numpy()[seg_of]
        perm, own = self.c.perm.numpy(), self.c.own_lens.numpy()
        pos, slots = np.zeros(T, np.int32), np.zeros(T, np.int64)
        for i, t in enumerate(perm):
            j = own[t] - 1
            pos[t] = pre[i] + j
            slots[t] = int(self.c.own_pages[t, j // self.page]) * self.page + j % self.page
        self.pos, self.slots = torch.from_numpy(pos), torch.from_numpy(slots)

    def device(self):
        d = {k: dev(v) for k, v in self.meta.items()}
        d.update(x=dev(self.x), k=dev(self.c.k), v=dev(self.c.v), A=dev(self.A), B=dev(self.B), Ao=dev(self.Ao),
                 Bo=dev(self.Bo), table=dev(self.table), qn=dev(self.qn), pos=dev(self.pos), slots=dev(self.slots),
                 pp=dev(self.c.prefix_pages), pl=dev(self.c.prefix_lens), op=dev(self.c.own_pages),
                 ol=dev(self.c.own_lens))
        d["wq"] = lm.linear_w4_prepare(dev(self.wqkv), dev(self.sqkv), dev(self.zqkv))
        d["wo"] = lm.linear_w4_prepare(dev(self.wo), dev(self.so))
        return d

    def run(self, d, ws=None):
        m = (d["indptr"], d["widx"], d["perm"], d["ranks"], d["sc"])
        y = lm.linear_w4(d["x"], d["wq"])
        lm.shrink_expand(d["x"], d["A"], d["B"], d["off"], *m, y, 3, self.R)
        q, k, v = _views(y, self.Hq, self.Hkv, self.D)
        q = lm.rope_append(q, k, v, d["table"], d["pos"], d["slots"], d["k"], d["v"], d["qn"], d["qn"], q_out=q)
        o = lm.prefix_attention(q, d["k"], d["v"], d["indptr"], d["perm"], d["pp"], d["pl"], d["op"], d["ol"],
                                self.c.scale, workspace=ws)
        z = lm.linear_w4(o, d["wo"])
        lm.shrink_expand(o, d["Ao"], d["Bo"], d["off_o"], *m, z, 1, self.R)
        return y, o, z


def test_decode_step():
    """Each operator on the values the one before it left, against the oracle on the same values."""
    s = Step(21)
    d = s.device()
    m = s.meta
    y0 = lm.linear_w4(d["x"], d["wq"])
    ref = oracle.linear_w4(s.x, s.wqkv, s.sqkv, s.zqkv)
    within(f64(y0), ref, dc.w4_bound("bf16", s.x, s.sqkv, ref, 64), "base")
    y, o, z = s.run(d)  # y holds the rotated q in place
    # the update and the rotation, from the base product as stored
    h = oracle.shrink(s.x, s.A, m["indptr"], m["widx"], m["perm"], m["ranks"], 3, s.R, "bf16")
    full = oracle.expand(h, s.B, m["off"], m["indptr"], m["widx"], m["perm"], m["ranks"], m["sc"], f64(y0), s.R, "bf16")
    qkv = torch.from_numpy(full).to(DT["bf16"])
    q, k, v = _views(qkv, s.Hq, s.Hkv, s.D)
    rq, rk, rv = oracle.rope_append(q, k, v, s.table, s.pos, s.slots, s.c.k, s.c.v, s.qn, s.qn)
    got_q = f64(y[:, :s.Hq * s.D])
    # the stored projection may differ by one step from the oracle's: 2 u relative of its elements,
    # which the norm (a factor of about 2 with its own sum) and the rotation (sqrt 2) carry on
    step = 8 * dc.U["bf16"] * np.abs(rq).reshape(s.T, s.Hq, s.D).max(2, keepdims=True)
    within(got_q.reshape(s.T, s.Hq, s.D), rq.reshape(s.T, s.Hq, s.D), step, "rotated q")
    stepk = 8 * dc.U["bf16"] * np.nanmax(np.abs(rk), axis=3, keepdims=True)
    within(f64(d["k"]), rk, stepk, "k cache")
    # attention and output, from the values as stored
    s.c.q, s.c.k, s.c.v = y[:, :s.Hq * s.D].cpu(), d["k"].cpu(), d["v"].cpu()
    aref, rl, spread = oracle.prefix_attention(*s.c.args())
    within(f64(o), aref, s.c.bounds(aref, rl, spread)[0], "attention")
    z0 = oracle.linear_w4(o.cpu(), s.wo, s.so)
    ho = oracle.shrink(o.cpu(), s.Ao, m["indptr"], m["widx"], m["perm"], m["ranks"], 1, s.R, "bf16")
    zref = oracle.expand(ho, s.Bo, m["off_o"], m["indptr"], m["widx"], m["perm"], m["ranks"], m["sc"], z0, s.R, "f64")
    # two roundings of the stored output (base, update) on top of the base product's own bound
    tol = dc.w4_bound("bf16", o.cpu(), s.so, z0, 128) + 2 * dc.U["bf16"] * (np.abs(z0) + np.abs(zref))
    within(f64(z), zref, tol + 4 * dc.U["bf16"] * np.abs(zref - z0), "output")


def test_decode_step_in_a_graph():
    """The step captured once and replayed: every replay gives the eager result of its own inputs, with
    eager work on the same operands between the replays, and two graphs sharing one workspace in
    turn."""
    s = Step(22)
    d = s.device()
    ws = lm.prefix_attention_workspace(d["x"].new_empty((s.T, s.Hq * s.D)), d["k"], d["indptr"], d["pp"], d["op"])
    s.run(d, ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run(d, ws))
        graphs.append(g)
    for r in range(3):
        d["x"].copy_(dc.normal(dc.gen(100 + r), (s.T, s.H), "bf16"))
        want = [t.clone() for t in s.run(d, ws)]
        torch.cuda.synchronize()
        for g, out in zip(graphs, outs):
            for t in out:
                t.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b), r


def test_decode_step_on_other_streams():
    """Two streams at once, each with its own workspace and cache: the results of one alone."""
    s = Step(23)
    want = [t.clone() for t in s.run(s.device())]
    sets = [s.device(), s.device()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for d, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(s.run(d))
    torch.cuda.synchronize()
    for out in got:
        for a, b in zip(out, want):
            assert torch.equal(a, b)
