"""The attention operators on the GPU against plain 64-bit implementations
(attn_ref.py, with the derivation of the tolerances), at the sizes, masks and
layouts where they can go wrong."""
import ctypes
import itertools
import math

import pytest
import torch

import all_reduce_residual_gb300 as arf
import attn_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ws():
    with arf.Workspace(0) as w:
        yield w
        torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def no_skipped_access(ws):
    """Every test leaves the counter of skipped accesses at zero; those that
    cause some read it themselves."""
    yield
    assert arf.bad_indices(ws) == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, dtype, seed, sigma=1.0):
    return (torch.randn(shape, generator=gen(seed)) * sigma).to(dtype)


def same(a, b):
    """Equal bits."""
    view = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().cpu().view(view), b.contiguous().cpu().view(view))


def inv_freq(rot, base=10000.0):
    return base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)


# ---- rotary ------------------------------------------------------------------


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(1, 1, 1, 2, 2), (1, 16, 4, 128, 128), (3, 5, 1, 64, 32), (7, 3, 3, 80, 32),
                                           (5, 2, 1, 96, 24), (2, 4, 2, 256, 256), (1, 1, 1, 13, 6), (33, 2, 2, 72, 16),
                                           (4865, 2, 1, 64, 64), (4866, 1, 2, 40, 16), (9, 40, 8, 128, 96)])
def test_rotary(ws, layout, T, Hq, Hk, D, rot):
    for dtype in (BF16, FP16):
        q, k = randn((T, Hq, D), dtype, 1), randn((T, Hk, D), dtype, 2)
        pos = torch.randint(-5, 200000, (T,), generator=gen(3), dtype=torch.int32)
        table = arf.RotaryTable(rot, layout=layout)
        qo, ko = arf.rotary(ws, q.to(DEV), k.to(DEV), pos.to(DEV), table)
        for got, x in ((qo, q), (ko, k)):
            want, bound = ref.rotate(x, pos, inv_freq(rot), rot, layout == "interleaved")
            ref.assert_close(got, want, bound + ref.half_step(want, dtype), f"{dtype}")
            assert same(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
def test_rotary_scaling_at_far_positions(ws, scaling, factor):
    rot, D = 64, 64
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 131071, 1000003], dtype=torch.int32)
    q = randn((len(pos), 3, D), BF16, 4)
    table = arf.RotaryTable(rot, base=500000.0, scaling=scaling, factor=factor, original_length=8192)
    w = inv_freq(rot, 500000.0 * (factor ** (rot / (rot - 2)) if scaling == "ntk" else 1.0))
    m = 1.0
    if scaling == "linear":
        w = w / factor
    if scaling == "yarn":
        keep = ((8192 * w / (2 * math.pi) - 1) / 31).clamp(0, 1)
        w, m = w * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1
    qo, ko = arf.rotary(ws, q.to(DEV), None, pos.to(DEV), table)
    assert ko is None
    want, bound = ref.rotate(q, pos, w, rot, False, m)
    # both sides hold w in binary64: an ulp or a few of it times the position
    ang = (pos.double().abs()[:, None] * w * 2.0 ** -49)[:, None, :].repeat(1, 1, 2)
    amp = q.double().abs().amax(-1, keepdim=True) * 2 * m
    ref.assert_close(qo, want, bound + ang * amp + ref.half_step(want, BF16))


def test_rotary_in_place_strided_and_unaligned(ws):
    T, D, rot = 37, 64, 32
    table = arf.RotaryTable(rot, layout="half")
    pos = torch.arange(T, dtype=torch.int32) * 11
    fused = randn((T, 6, D), FP16, 5)  # 4 query heads, 2 key heads, and the space behind a slice
    want, bound = ref.rotate(fused, pos, inv_freq(rot), rot, False)
    bound = bound + ref.half_step(want, FP16)
    x = fused.to(DEV)
    q, k = x[:, :4], x[:, 4:]
    qo, ko = arf.rotary(ws, q, k, pos.to(DEV), table, q_out=q, k_out=k)
    assert qo is q and ko is k
    ref.assert_close(x, want, bound, "in place")
    # heads outermost, and an odd element offset (2-byte aligned only)
    y = torch.zeros(6 * T * D + 1, dtype=FP16, device=DEV)
    z = y[1:].view(6, T, D).transpose(0, 1)
    z.copy_(fused)
    out = torch.full((T, 9, D + 8), 7.0, dtype=FP16, device=DEV)
    arf.rotary(ws, z, None, pos.to(DEV), table, q_out=out[:, 1:7, 3:3 + D])
    ref.assert_close(out[:, 1:7, 3:3 + D], want, bound, "unaligned")
    rest = out.clone()
    rest[:, 1:7, 3:3 + D] = 7.0
    assert bool((rest == 7.0).all()), "wrote outside q_out"


def test_rotary_keeps_special_values(ws):
    q = torch.zeros(1, 1, 32, dtype=BF16)
    q[0, 0, 0], q[0, 0, 5], q[0, 0, 20] = math.inf, math.nan, -0.0
    table = arf.RotaryTable(16)
    qo, _ = arf.rotary(ws, q.to(DEV), None, torch.tensor([3], dtype=torch.int32, device=DEV), table)
    want, _ = ref.rotate(q, torch.tensor([3]), inv_freq(16), 16, False)
    assert torch.equal(qo.cpu().double().isnan(), want.isnan()) and same(qo[..., 16:], q[..., 16:])
    assert torch.equal(qo.cpu().double().isinf(), want.isinf())


def test_rotary_of_nothing(ws):
    e = torch.empty(0, 4, 64, dtype=BF16, device=DEV)
    qo, ko = arf.rotary(ws, e, e, torch.empty(0, dtype=torch.int32, device=DEV), arf.RotaryTable(64))
    assert qo.shape == e.shape and ko.shape == e.shape


def test_rotary_wrapper_refuses(ws):
    q = torch.zeros(2, 4, 64, dtype=BF16, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    t = arf.RotaryTable(64)
    for a in ((q.float(), None, pos), (q, None, pos.long()), (q, None, pos[:1]), (q, None, pos.cpu()),
              (q.cpu(), None, pos), (q, q.half(), pos), (q, q[:1], pos), (q[0], None, pos),
              (q.transpose(1, 2), None, pos)):
        with pytest.raises(ValueError):
            arf.rotary(ws, *a, t)
    with pytest.raises(arf.ArfError):
        arf.rotary(ws, q[..., :32].contiguous(), None, pos, t)


# ---- append ------------------------------------------------------------------


def pages(n, size, heads, D, dtype, layout, seed, scale=1.0):
    shape = (n, size, heads, D) if layout == "nhd" else (n, heads, size, D)
    if dtype == E4M3:
        return (torch.randn(shape, generator=gen(seed)) / scale).clamp(-448, 448).to(E4M3)
    return torch.randn(shape, generator=gen(seed)).to(dtype)


def pick(x, at):
    """x[at]; torch does not index 8-bit floats on the CPU."""
    return x.view(torch.uint8)[at].view(E4M3) if x.dtype == E4M3 else x[at]


def at_slots(p, layout):
    """[slots, heads, D] of page tensors."""
    x = p.view(torch.uint8) if p.dtype == E4M3 else p
    x = (x.transpose(1, 2) if layout == "hnd" else x).contiguous()
    return (x.view(E4M3) if p.dtype == E4M3 else x).reshape(-1, x.shape[2], x.shape[3])


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,page", [(1, 8, 2, 128, 128, 16), (5, 3, 1, 64, 32, 1), (19, 4, 4, 80, 16, 7),
                                                (6, 2, 2, 40, 20, 3), (4900, 2, 1, 64, 64, 64), (3, 5, 1, 13, 4, 5)])
def test_append(ws, layout, e4m3, T, Hq, Hk, D, rot, page):
    for dtype, interleaved in ((BF16, False), (FP16, True)):
        ks, vs = (0.02, 0.013) if e4m3 else (1.0, 1.0)
        cdt = E4M3 if e4m3 else dtype
        q, k, v = (randn((T, h, D), dtype, i) for i, h in enumerate((Hq, Hk, Hk)))
        n = -(-T // page) + 2
        kp, vp = pages(n, page, Hk, D, cdt, layout, 8, ks), pages(n, page, Hk, D, cdt, layout, 9, vs)
        kd, vd = kp.to(DEV), vp.to(DEV)
        cache = arf.KVCache(kd, vd, layout, ks, vs)
        pos = torch.randint(0, 5000, (T,), generator=gen(10), dtype=torch.int32)
        slots = torch.randperm(n * page, generator=gen(11))[:T]
        if T > 2:
            slots[1] = -1
        table = arf.RotaryTable(rot, layout="interleaved" if interleaved else "half")
        qo = arf.rotary_append(ws, q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), slots.to(DEV), table, cache)
        want, bound = ref.rotate(q, pos, inv_freq(rot), rot, interleaved)
        ref.assert_close(qo, want, bound + ref.half_step(want, dtype), "q")
        assert same(qo[..., rot:], q[..., rot:])
        kept = slots >= 0
        kr, kb = ref.rotate(k, pos, inv_freq(rot), rot, interleaved)
        for got, before, x, xb, scale in ((kd, kp, kr, kb, ks), (vd, vp, v.double(), torch.zeros(()), vs)):
            got, before = at_slots(got.cpu(), layout), at_slots(before, layout)
            rest = torch.ones(n * page, dtype=torch.bool)
            rest[slots[kept]] = False
            assert same(pick(got, rest), pick(before, rest)), "a slot that no token names changed"
            y = (x / scale).clamp(-448, 448)[kept]
            xb = (xb / scale + x.abs() / scale * 2.0 ** -22 if e4m3 else xb).expand(x.shape)[kept]
            # the bound on the value before its rounding moves it at most by
            # as much, and to the next of the type's values
            ref.assert_close(pick(got, slots[kept]), y, xb * 1.07 + ref.half_step(y.abs() + xb, cdt), "cache")
        if not e4m3:
            assert same(at_slots(vd.cpu(), layout)[slots[kept]], v[kept])


def test_append_without_rotation_or_queries(ws):
    T, H, D = 9, 2, 64
    k, v = randn((T, H, D), BF16, 1), randn((T, H, D), BF16, 2)
    kd, vd = (torch.zeros(3, 4, H, D, dtype=BF16, device=DEV) for _ in range(2))
    cache = arf.KVCache(kd, vd)
    slots = torch.arange(2, 2 + T)
    assert arf.rotary_append(ws, None, k.to(DEV), v.to(DEV), None, slots.to(DEV), None, cache) is None
    for got, x in ((kd, k), (vd, v)):
        got = at_slots(got.cpu(), "nhd")
        assert same(got[2:2 + T], x) and not got[:2].any() and not got[2 + T:].any()
    pos = torch.arange(T, dtype=torch.int32)
    arf.rotary_append(ws, None, k.to(DEV), v.to(DEV), pos.to(DEV), slots.to(DEV), arf.RotaryTable(D), cache)
    want, bound = ref.rotate(k, pos, inv_freq(D), D, False)
    ref.assert_close(at_slots(kd.cpu(), "nhd")[2:2 + T], want, bound + ref.half_step(want, BF16))


def test_append_skips_slots_out_of_range(ws):
    T, H, D = 70, 1, 64
    k, v = randn((T, H, D), FP16, 1), randn((T, H, D), FP16, 2)
    kd, vd = (torch.zeros(5, 16, H, D, dtype=FP16, device=DEV) for _ in range(2))
    slots = torch.arange(T)
    slots[3], slots[40], slots[41], slots[69] = 80, 2 ** 62, -2 ** 63, 1 << 32
    arf.rotary_append(ws, None, k.to(DEV), v.to(DEV), None, slots.to(DEV), None, arf.KVCache(kd, vd))
    assert arf.bad_indices(ws) == 3  # the negative one is padding
    good = (slots >= 0) & (slots < 80)
    got = at_slots(vd.cpu(), "nhd")
    assert same(got[slots[good]], v[good])
    assert not got[[3, 40, 41, 69]].any() and not got[70:].any()


def test_append_saturates_e4m3(ws):
    v = torch.tensor([0.0, -0.0, 447.0, 449.0, 463.9, 464.0, 1e4, -1e4, math.inf, -math.inf, math.nan, 2.0 ** -10,
                      2.0 ** -9, 3 * 2.0 ** -10, -17.0, 0.3], dtype=BF16).view(1, 1, 16)
    kd, vd = (torch.zeros(1, 1, 1, 16, dtype=E4M3, device=DEV) for _ in range(2))
    arf.rotary_append(ws, None, v.to(DEV), v.to(DEV), None, torch.zeros(1, dtype=torch.long, device=DEV), None,
                      arf.KVCache(kd, vd))
    want = v.float().clamp(-448, 448).to(E4M3).float().view(-1)
    for got in (kd, vd):
        got = got.cpu().float().view(-1)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0), want.nan_to_num(0))


def test_append_past_32_bit_offsets(ws):
    """A cache whose last page begins beyond 2^32 elements."""
    D, far = 64, (1 << 32) + 64
    base = torch.zeros(far + 2 * D, dtype=BF16, device=DEV)
    kd = base.as_strided((2, 1, 1, D), (far, D, D, 1))
    vd = base.as_strided((2, 1, 1, D), (far, D, D, 1), D)
    k, v = randn((2, 1, D), BF16, 1).to(DEV), randn((2, 1, D), BF16, 2).to(DEV)
    cache = arf.KVCache(kd, vd)
    arf.rotary_append(ws, None, k, v, None, torch.tensor([1, 0], device=DEV), None, cache)
    assert same(kd[1, 0], k[0]) and same(vd[0, 0], v[1])
    q = randn((1, 2, D), BF16, 3)
    table = torch.tensor([[0, 1]], dtype=torch.int32)
    lens = torch.tensor([2], dtype=torch.int32)
    got = arf.paged_decode(ws, q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    want = ref.decode(q, kd.cpu().contiguous(), vd.cpu().contiguous(), "nhd", table, lens, D ** -0.5)
    ref.assert_decode(got, want, BF16)
    arf.copy_pages(ws, cache, [1], [0])
    assert same(kd[0], kd[1]) and same(vd[0], vd[1])


# ---- decode ------------------------------------------------------------------


def batch(lens, page, Hkv, G, D, dtype, cdt, layout, seed=0, width=None, ks=1.0, vs=1.0, nan=True):
    """Queries, pages in random order with NaN in every row no sequence holds,
    and the table (-1 behind a sequence's end)."""
    g = gen(seed)
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    kp, vp = pages(total, page, Hkv, D, cdt, layout, seed + 1, ks), pages(total, page, Hkv, D, cdt, layout, seed + 2, vs)
    order = torch.randperm(total, generator=g).to(torch.int32)
    width = max(need + [1]) if width is None else width
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    held = torch.zeros(total, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        table[b, : need[b]] = order[at:at + need[b]]
        for i in range(need[b]):
            held[table[b, i], : min(page, n - i * page)] = True
        at += need[b]
    if nan:
        for p in (kp, vp):
            x = p.view(torch.uint8) if cdt == E4M3 else p
            x = x if layout == "nhd" else x.transpose(1, 2)
            x[~held] = 0x7F if cdt == E4M3 else math.nan
    q = randn((len(lens), Hkv * G, D), dtype, seed + 3, 2.0)
    return q, kp, vp, table, torch.tensor(lens, dtype=torch.int32)


def check(ws, lens, page=16, Hkv=2, G=4, D=128, dtype=BF16, cdt=None, layout="nhd", cap=0.0, window=0, seed=0,
          width=None):
    cdt = dtype if cdt is None else cdt
    ks, vs = (0.02, 0.013) if cdt == E4M3 else (1.0, 1.0)
    q, kp, vp, table, n = batch(lens, page, Hkv, G, D, dtype, cdt, layout, seed, width=width, ks=ks, vs=vs)
    cache = arf.KVCache(kp.to(DEV), vp.to(DEV), layout, ks, vs)
    args = (ws, q.to(DEV), cache, table.to(DEV), n.to(DEV))
    got = arf.paged_decode(*args, softcap=cap, window=window)
    want = ref.decode(q, kp, vp, layout, table, n, D ** -0.5, cap, window, ks, vs)
    what = f"page={page} Hkv={Hkv} G={G} D={D} {dtype} {cdt} {layout} cap={cap} window={window}"
    ref.assert_decode(got, want, dtype, what)
    again = arf.paged_decode(*args, softcap=cap, window=window)
    assert same(got[0], again[0]) and same(got[1], again[1]), f"{what}: two equal calls differ"


LENS = [0, 1, 2, 15, 16, 17, 0, 31, 33, 63, 64, 65, 127, 128, 129, 200, 513, 0]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"])
@pytest.mark.parametrize("G", [1, 3, 8, 11, 16, 20])
def test_decode_types_and_groups(ws, D, kind, G):
    dtype = BF16 if kind.startswith("bf16") else FP16
    check(ws, LENS, D=D, G=G, Hkv=2, dtype=dtype, cdt=E4M3 if "e4m3" in kind else dtype, seed=G)


@pytest.mark.parametrize("page,layout,Hkv", [(1, "nhd", 1), (3, "hnd", 2), (7, "nhd", 4), (16, "hnd", 1), (64, "nhd", 8),
                                             (100, "hnd", 3), (256, "nhd", 2), (1024, "hnd", 1)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_pages_and_layouts(ws, page, layout, Hkv, e4m3):
    check(ws, LENS, page=page, layout=layout, Hkv=Hkv, G=2, cdt=E4M3 if e4m3 else BF16, seed=page)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 64, 100, 512, 513, 10000])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_decode_window_and_cap(ws, window, cap):
    check(ws, LENS, window=window, cap=cap, seed=window)
    check(ws, LENS, window=window, cap=cap, D=256, G=1, dtype=FP16, cdt=E4M3, layout="hnd", seed=window)


@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [5000], [20011, 3, 0, 777], [1] * 300, [0] * 200 + [70] * 150,
                                  list(range(0, 260)), [40000]])
def test_decode_splits(ws, lens):
    check(ws, lens, Hkv=1, G=8, page=16)
    check(ws, lens, Hkv=1, G=3, D=64, page=32, cdt=E4M3)


@pytest.mark.parametrize("tokens", [1, 16, 64, 65, 128, 129, 256, 300, 512, 1024, 2048, 2049])
@pytest.mark.parametrize("cap,window", [(0.0, 0), (7.0, 100)])
def test_decode_short_and_long_forms(ws, tokens, cap, window):
    """Around the table widths at which the split changes: clusters of 1 to 8
    CTAs, then the whole device."""
    lens = [tokens, 1, 0, tokens // 2, max(1, tokens - 1)]
    check(ws, lens, page=16, G=4, Hkv=2, cap=cap, window=window)
    check(ws, lens, page=8, G=12, Hkv=1, D=64, dtype=FP16, cdt=E4M3, cap=cap, window=window)
    check(ws, lens, page=64, G=9, Hkv=1, D=256, layout="hnd", cap=cap, window=window)


def test_decode_scratch(ws):
    """No scratch for short tables; scratch elsewhere, refused when too small."""
    q, kp, vp, table, n = (x.to(DEV) for x in batch([9000, 3], 16, 2, 2, 64, BF16, BF16, "nhd",
                                                          width=10000))
    cache = arf.KVCache(kp, vp)
    size = ctypes.c_size_t()
    need = lambda width, window: (arf.arf_paged_decode_scratch_bytes(  # noqa: E731
        ws.handle, cache.struct, 2, 4, width, window, size), size.value)
    assert need(4, 0) == (arf.ARF_OK, 0) and need(100000, 64) == (arf.ARF_OK, 0) and need(0, 0) == (arf.ARF_OK, 0)
    st, wide = need(table.shape[1], 0)
    assert st == arf.ARF_OK and wide > 0
    for bad in ((-1, 0), (4, -1)):
        assert need(*bad)[0] == arf.ARF_ERR_INVALID_ARG
    out, lse = torch.full_like(q, 5.0), torch.zeros(2, 4, device=DEV)
    scratch = torch.empty(wide, dtype=torch.uint8, device=DEV)
    heads = lambda x: arf.Heads(x.data_ptr(), x.stride(0), x.stride(1), x.shape[1])  # noqa: E731
    call = lambda ptr, nbytes: arf.arf_paged_decode(  # noqa: E731
        ws.handle, cache.struct, 2, arf.ARF_BF16, heads(q), table.data_ptr(), table.stride(0), table.shape[1],
        n.data_ptr(), 0.125, 0.0, 0, heads(out), lse.data_ptr(), ptr, nbytes, torch.cuda.current_stream().cuda_stream)
    assert call(scratch.data_ptr(), wide - 1) == arf.ARF_ERR_INVALID_ARG
    assert call(None, wide) == arf.ARF_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((out == 5.0).all()), "a refused call wrote its output"
    assert call(scratch.data_ptr(), wide) == arf.ARF_OK
    ref.assert_decode((out, lse), ref.decode(q.cpu(), kp.cpu(), vp.cpu(), "nhd", table.cpu(), n.cpu(), 0.125), BF16)


@pytest.mark.parametrize("width", [None, 300])
def test_decode_many_sequences(ws, width):
    """More short items than CTAs: a warp per item, and, with a wide table,
    the dealt form with more sequences than a CTA has threads."""
    check(ws, [(7 * i) % 23 for i in range(1100)], Hkv=1, G=1, D=64, page=8, width=width)
    check(ws, [(5 * i) % 61 for i in range(210)], Hkv=2, G=12, D=128, page=7, window=33, width=width)
    check(ws, [(3 * i) % 33 for i in range(330)], Hkv=1, G=5, D=256, page=16, cap=9.0, dtype=FP16, width=width)
    check(ws, [(11 * i) % 90 for i in range(500)], Hkv=2, G=9, D=64, page=16, cdt=E4M3, layout="hnd", width=width)
    check(ws, [(13 * i) % 130 for i in range(700)], Hkv=1, G=2, D=128, page=32, cdt=E4M3, dtype=FP16, window=100,
          width=width)


def test_decode_many_short_sequences_with_bad_entries(ws):
    q, kp, vp, table, n = batch([(3 * i) % 40 for i in range(400)], 16, 1, 2, 64, BF16, BF16, "nhd", nan=False)
    table[5, 0], table[7, 1] = kp.shape[0], -3
    n[9], n[11] = -1, 10 ** 6
    table[11] = torch.arange(table.shape[1], dtype=torch.int32)
    got = arf.paged_decode(ws, q.to(DEV), arf.KVCache(kp.to(DEV), vp.to(DEV)), table.to(DEV), n.to(DEV))
    assert arf.bad_indices(ws) > 0
    ref.assert_decode(got, ref.decode(q, kp, vp, "nhd", table, n, 0.125, skip_bad=True), BF16)


def test_decode_large_scores(ws):
    """Scores in the hundreds: one token takes everything; then equal scores."""
    q, kp, vp, table, n = batch([300, 77], 16, 1, 4, 128, BF16, BF16, "nhd")
    for q in (q * 64, q * 0):
        got = arf.paged_decode(ws, q.to(DEV), arf.KVCache(kp.to(DEV), vp.to(DEV)), table.to(DEV), n.to(DEV))
        ref.assert_decode(got, ref.decode(q, kp, vp, "nhd", table, n, 128 ** -0.5), BF16)
    # keys and values at the type's limits, queries far below an e4m3 cache's fp16 products
    for sigma in (2.0 ** -100, 2.0 ** 60):
        q, kp, vp, table, n = batch([65, 9], 16, 1, 2, 64, BF16, E4M3, "nhd", ks=1.0, vs=1.0)
        q = (q.float() * sigma).to(BF16)
        scale = 0.1 / sigma
        got = arf.paged_decode(ws, q.to(DEV), arf.KVCache(kp.to(DEV), vp.to(DEV)), table.to(DEV), n.to(DEV), scale=scale)
        ref.assert_decode(got, ref.decode(q, kp, vp, "nhd", table, n, scale), BF16, f"sigma={sigma}")


@pytest.mark.parametrize("cap", [0.05, 1.0, 300.0, 1e5, 1e30])
def test_decode_cap_sizes(ws, cap):
    """Caps far below and far above the scores (the bound: a relative error of
    2^-20 of the score, as for the scores themselves with A = |s|)."""
    q, kp, vp, table, n = batch([300, 77, 5], 16, 1, 4, 64, FP16, FP16, "nhd")
    got = arf.paged_decode(ws, q.to(DEV), arf.KVCache(kp.to(DEV), vp.to(DEV)), table.to(DEV), n.to(DEV), softcap=cap)
    out, lse, tol, ltol = ref.decode(q, kp, vp, "nhd", table, n, 0.125, softcap=cap)
    s = torch.einsum("bhd,phd->bhp", q.double(), kp.double().flatten(0, 1)[:, :1].repeat(1, 4, 1).nan_to_num(0))
    e_s = min(cap, float(s.abs().max()) * 0.125) * 2.0 ** -20
    bare = ref.decode(q, kp, vp, "nhd", table, n, 0.125, softcap=cap, cap_error=0.0)
    spread = float(vp.double().nan_to_num(0).abs().max())
    ref.assert_close(got[0], out, bare[2] + math.expm1(2 * e_s) * 2 * spread + ref.half_step(out, FP16), "out")
    ref.assert_close(got[1], lse, bare[3] + 2 * e_s, "lse")


def test_decode_many_small_weights_in_fp16(ws):
    """One token far above 30000 equal ones, whose weights of 2^-15 each sum
    to as much as it has: they must not be rounded as fp16 subnormals."""
    n, D = 30001, 64
    k = torch.zeros(-(-n // 64), 64, 1, D, dtype=FP16)
    v = torch.ones_like(k)
    q = torch.zeros(1, 1, D, dtype=FP16)
    q[..., 0] = 1.0
    k[0, 0, 0, 0] = 8.0 * (15.3 * math.log(2.0))
    v[0, 0] = -1.0
    table = torch.arange(k.shape[0], dtype=torch.int32)[None]
    lens = torch.tensor([n], dtype=torch.int32)
    got = arf.paged_decode(ws, q.to(DEV), arf.KVCache(k.to(DEV), v.to(DEV)), table.to(DEV), lens.to(DEV))
    ref.assert_decode(got, ref.decode(q, k, v, "nhd", table, lens, 0.125), FP16)


def test_decode_infinities(ws):
    """-inf scores are masked out; +inf or NaN scores and values give NaN where
    the definition does, and only there."""
    q, kp, vp, table, n = batch([40, 20, 33, 70], 16, 1, 2, 64, FP16, FP16, "nhd", nan=False)
    q[:, :, 0] = 1.0
    tok = lambda b, j: (int(table[b, j // 16]), j % 16, 0)  # noqa: E731
    kp[tok(0, 5)][0] = -math.inf          # masked
    for j in range(20):                   # no score left
        kp[tok(1, j)][0] = -math.inf
    kp[tok(2, 7)][0] = math.inf           # the whole row is NaN
    vp[tok(3, 69)][3] = math.inf          # one element of out
    got = arf.paged_decode(ws, q.to(DEV), arf.KVCache(kp.to(DEV), vp.to(DEV)), table.to(DEV), n.to(DEV))
    out, lse = (x.cpu() for x in got)
    assert not out[1].any() and bool((lse[1] == -math.inf).all())
    assert bool(out[2].isnan().all()) and bool(lse[2].isnan().all())
    assert bool((out[3, :, 3] == math.inf).all()) and bool(out[3, :, :3].isfinite().all())
    vp[tok(3, 69)][3] = 0.0
    kp[tok(0, 5)][0] = -2.0 ** 15  # a score of about -4000: also nothing
    want = ref.decode(q, kp, vp, "nhd", table, n, 0.125)
    ref.assert_close(out[0], want[0][0], want[2][0] + ref.half_step(want[0][0], FP16) + 1e-30)


def test_decode_strided_tensors(ws):
    """Queries inside a fused projection, out inside a larger tensor, keys and
    values interleaved per page, a table inside a wider one."""
    lens, page, Hkv, G, D = [33, 0, 100, 17], 16, 2, 4, 64
    q, kp, vp, table, n = batch(lens, page, Hkv, G, D, BF16, BF16, "nhd")
    both = torch.stack((kp, vp), 1).to(DEV)  # [pages, 2, page, heads, D]
    cache = arf.KVCache(both[:, 0], both[:, 1])
    fused = torch.zeros(4, Hkv * G + 5, D, dtype=BF16, device=DEV)
    fused[:, 2:2 + Hkv * G] = q.to(DEV)
    wide = torch.full((4, table.shape[1] + 9), -7, dtype=torch.int32, device=DEV)
    wide[:, 4:4 + table.shape[1]] = table.to(DEV)
    big = torch.full((4, Hkv * G + 1, D + 8), 3.0, dtype=BF16, device=DEV)
    out = big[:, :Hkv * G, :D]
    got = arf.paged_decode(ws, fused[:, 2:2 + Hkv * G], cache, wide[:, 4:4 + table.shape[1]], n.to(DEV), out=out)
    assert got[0] is out
    want = ref.decode(q, kp, vp, "nhd", table, n, D ** -0.5)
    ref.assert_decode(got, want, BF16)
    assert bool((big[:, Hkv * G:] == 3.0).all()) and bool((big[..., D:] == 3.0).all())
    # one table row for all sequences
    same_n = torch.tensor([33, 0, 5, 17], dtype=torch.int32)
    row = table[:1].to(DEV).expand(4, -1)
    cached = (kp.to(DEV), vp.to(DEV))
    ref.assert_decode(arf.paged_decode(ws, q.to(DEV), arf.KVCache(*cached), row, same_n.to(DEV)),
                      ref.decode(q, kp, vp, "nhd", table[:1].expand(4, -1), same_n, D ** -0.5), BF16)
    # heads of a shard inside a cache that holds more
    wide_k = torch.randn(kp.shape[0], page, 5, D, generator=gen(4)).to(BF16)
    wide_v = torch.randn(kp.shape[0], page, 5, D, generator=gen(5)).to(BF16)
    wide_k[:, :, 1:3], wide_v[:, :, 1:3] = kp, vp
    cache = arf.KVCache(wide_k.to(DEV)[:, :, 1:3], wide_v.to(DEV)[:, :, 1:3])
    ref.assert_decode(arf.paged_decode(ws, q.to(DEV), cache, table.to(DEV), n.to(DEV)), want, BF16)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-30])
def test_decode_scales_and_broadcast_inputs(ws, scale):
    """Any finite softmax scale; one query for all heads, one key head for all
    (strides of 0)."""
    q, kp, vp, table, n = batch([70, 5, 0, 300], 16, 1, 6, 64, BF16, BF16, "nhd", nan=False)
    q = q[:, :1].expand(-1, 6, -1)
    kd, vd = kp.to(DEV).expand(-1, -1, 2, -1), vp.to(DEV).expand(-1, -1, 2, -1)
    got = arf.paged_decode(ws, q.to(DEV)[:, :1].expand(-1, 6, -1), arf.KVCache(kd, vd), table.to(DEV), n.to(DEV),
                           scale=scale)
    ref.assert_decode(got, ref.decode(q, kp.expand(-1, -1, 2, -1), vp.expand(-1, -1, 2, -1), "nhd", table, n, scale),
                      BF16)


def test_decode_skips_bad_pages_and_lengths(ws):
    page = 16
    q, kp, vp, table, n = batch([100, 64, 30, 40], page, 2, 2, 128, BF16, BF16, "nhd", nan=False)
    table[0, 2] = kp.shape[0]      # one page out of range
    table[0, 5] = -1
    table[1, :] = -2 ** 31         # a sequence without one page in range
    n[2] = -5                      # taken as 0
    n[3] = 10 ** 9                 # taken as the table's width
    table[3, :] = torch.arange(table.shape[1], dtype=torch.int32)
    got = arf.paged_decode(ws, q.to(DEV), arf.KVCache(kp.to(DEV), vp.to(DEV)), table.to(DEV), n.to(DEV))
    assert arf.bad_indices(ws) > 0
    ref.assert_decode(got, ref.decode(q, kp, vp, "nhd", table, n, 128 ** -0.5, skip_bad=True), BF16)


def test_decode_shared_pages_and_empty_calls(ws):
    q, kp, vp, table, n = batch([50, 50, 0], 16, 2, 2, 64, BF16, BF16, "nhd")
    table[1] = table[0]  # a fork: the same pages twice
    cache = arf.KVCache(kp.to(DEV), vp.to(DEV))
    got = arf.paged_decode(ws, q.to(DEV), cache, table.to(DEV), n.to(DEV))
    ref.assert_decode(got, ref.decode(q, kp, vp, "nhd", table, n, 0.125), BF16)
    out, lse = arf.paged_decode(ws, q[:0].to(DEV), cache, table[:0].to(DEV), n[:0].to(DEV))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = arf.paged_decode(ws, q.to(DEV), cache, table[:, :0].to(DEV), torch.zeros_like(n).to(DEV))
    assert not out.any() and bool((lse == -math.inf).all())


def test_decode_wrapper_refuses(ws):
    q, kp, vp, table, n = (x.to(DEV) for x in batch([50, 3], 16, 2, 2, 64, BF16, BF16, "nhd"))
    cache = arf.KVCache(kp, vp)
    for a in ((q.float(), cache, table, n), (q[:, :3], cache, table, n), (q, cache, table.long(), n),
              (q, cache, table, n.long()), (q, cache, table, n[:1]), (q, cache, table[:1], n),
              (q.cpu(), cache, table, n), (q, cache, table.t().contiguous().t(), n), (q, cache, table.cpu(), n)):
        with pytest.raises(ValueError):
            arf.paged_decode(ws, *a)
    for kw in (dict(out=q[:1]), dict(lse=torch.empty(2, 4, device=DEV, dtype=BF16)), dict(out=q.half())):
        with pytest.raises(ValueError):
            arf.paged_decode(ws, q, cache, table, n, **kw)
    for kw in (dict(window=-1), dict(softcap=-1.0), dict(scale=math.nan)):
        with pytest.raises(arf.ArfError):
            arf.paged_decode(ws, q, cache, table, n, **kw)
    for handle in (arf.RotaryTable(64), None, kp):
        with pytest.raises(ValueError):
            arf.paged_decode(ws, q, handle, table, n)
    with pytest.raises(ValueError):
        arf.rotary(ws, q, None, n, cache)
    with pytest.raises(ValueError):
        arf.rotary(ws, q, None, n, arf.RotaryTable(64, device="cpu"))
    with pytest.raises(arf.ArfError):  # fp16 queries on a bf16 cache
        arf.paged_decode(ws, q.half(), cache, table, n)
    odd = torch.zeros(2, 4, 72, dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        arf.paged_decode(ws, odd, cache, table, n)


# ---- streams and graphs --------------------------------------------------------


def test_decode_on_another_stream(ws):
    q, kp, vp, table, n = batch([700, 50, 90], 16, 2, 4, 128, BF16, BF16, "nhd")
    want = ref.decode(q, kp, vp, "nhd", table, n, 128 ** -0.5)
    cache = arf.KVCache(kp.to(DEV), vp.to(DEV))
    q, table, n = q.to(DEV), table.to(DEV), n.to(DEV)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(20):
        got = [arf.paged_decode(ws, q, cache, table, n, stream=s) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        ref.assert_decode(g, want, BF16)


@pytest.mark.parametrize("width", [6, 700])
def test_captured_steps_share_a_workspace(ws, width):
    """Two graphs of append and decode on one workspace, replayed at the same
    time, with lengths, slots and positions that change between replays; a
    short table (clusters) and a wide one (scratch)."""
    page, Hkv, G, D, B = 16, 2, 4, 64, 3
    states = []
    for k in range(2):
        q, kp, vp, table, n = batch([60, 33, 5], page, Hkv, G, D, BF16, BF16, "nhd", seed=10 * k, width=width, nan=False)
        free = [p for p in range(kp.shape[0]) if p not in table]
        table[0, 4] = free[0]  # room for one more page
        kn, vn = randn((B, Hkv, D), BF16, 50 + k), randn((B, Hkv, D), BF16, 60 + k)
        dev = dict(q=q.to(DEV), k=kn.to(DEV), v=vn.to(DEV), kp=kp.to(DEV), vp=vp.to(DEV), table=table.to(DEV),
                   lens=n.to(DEV), slots=torch.full((B,), -1, device=DEV), pos=torch.zeros(B, dtype=torch.int32, device=DEV))
        states.append((dev, dict(q=q, k=kn, v=vn, kp=kp, vp=vp, table=table, lens=n)))
    rot = arf.RotaryTable(D)
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []

    def step(d):
        q = arf.rotary_append(ws, d["q"], d["k"], d["v"], d["pos"], d["slots"], rot, arf.KVCache(d["kp"], d["vp"]))
        return arf.paged_decode(ws, q, arf.KVCache(d["kp"], d["vp"]), d["table"], d["lens"])

    for s, (d, _) in zip(streams, states):
        step(d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(step(d))
        graphs.append(g)
    for it in range(6):
        for s, g, (d, h) in zip(streams, graphs, states):
            h["lens"] += 1
            at = h["lens"].long() - 1
            pages_ = h["table"].gather(1, (at // page)[:, None])[:, 0].long()
            slots = pages_ * page + at % page
            pos = at.to(torch.int32)
            d["lens"].copy_(h["lens"])
            d["slots"].copy_(slots)
            d["pos"].copy_(pos)
            h["slots"], h["pos"] = slots, pos
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (d, h), got in zip(states, outs):
            flat_k, flat_v = h["kp"].view(-1, Hkv, D), h["vp"].view(-1, Hkv, D)
            want_k, kb = ref.rotate(h["k"], h["pos"], inv_freq(D), D, False)
            new_k = at_slots(d["kp"].cpu(), "nhd")[h["slots"]]
            ref.assert_close(new_k, want_k, kb + ref.half_step(want_k, BF16))
            flat_k[h["slots"]], flat_v[h["slots"]] = new_k, h["v"]  # as stored
            assert same(d["kp"], h["kp"]) and same(d["vp"], h["vp"])
            q = arf.rotary(ws, d["q"], None, d["pos"], rot)[0].cpu()
            ref.assert_decode(got, ref.decode(q, h["kp"], h["vp"], "nhd", h["table"], h["lens"], D ** -0.5), BF16)


def test_captured_copy_and_rotary(ws):
    k = torch.randn(12, 4, 2, 64, generator=gen(1)).to(BF16).to(DEV)
    v = torch.randn(12, 4, 2, 64, generator=gen(2)).to(BF16).to(DEV)
    cache = arf.KVCache(k, v)
    q = randn((5, 3, 64), BF16, 3).to(DEV)
    pos = torch.zeros(5, dtype=torch.int32, device=DEV)
    table = arf.RotaryTable(64)
    arf.rotary(ws, q, None, pos, table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        arf.copy_pages(ws, cache, [1, 2], [7, 8])
        out, _ = arf.rotary(ws, q, None, pos, table)
    for it in range(3):
        k.copy_(torch.randn(k.shape, generator=gen(10 + it)).to(BF16))
        pos.fill_(it * 1000)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same(k[7:9], k[1:3]) and same(v[7:9], v[1:3])
        want, bound = ref.rotate(q.cpu(), pos.cpu(), inv_freq(64), 64, False)
        ref.assert_close(out, want, bound + ref.half_step(want, BF16))


def test_calls_from_two_threads(ws):
    """Two threads on one workspace, each on a stream of its own."""
    import threading
    errors = []

    def work(seed):
        try:
            q, kp, vp, table, n = batch([5000, 17, 0, 300], 16, 1, 4, 64, BF16, BF16, "nhd", seed=seed)
            want = ref.decode(q, kp, vp, "nhd", table, n, 0.125)
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                dev = [x.to(DEV) for x in (q, kp, vp, table, n)]
                cache = arf.KVCache(dev[1], dev[2])
                for _ in range(50):
                    got = arf.paged_decode(ws, dev[0], cache, dev[3], dev[4])
                s.synchronize()
                ref.assert_decode(got, want, BF16)
        except Exception as e:  # noqa: BLE001  (reported by the test's thread)
            errors.append(e)
    ts = [threading.Thread(target=work, args=(100 * i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not errors, errors


def test_closed_workspace_and_empty_cache(ws):
    q = torch.zeros(2, 4, 64, dtype=BF16, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    none = torch.zeros(0, 16, 2, 64, dtype=BF16, device=DEV)
    cache = arf.KVCache(none, none)
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    out, lse = arf.paged_decode(ws, q + 1, cache, table, pos)
    assert not out.any() and bool((lse == -math.inf).all())
    k = q[:, :2].contiguous()
    arf.rotary_append(ws, None, k, k, None, torch.full((2,), -1, device=DEV), None, cache)
    arf.rotary_append(ws, None, k, k, None, torch.zeros(2, dtype=torch.long, device=DEV), None, cache)
    assert arf.bad_indices(ws) == 2
    arf.copy_pages(ws, cache, [], [])
    closed = arf.Workspace(0)
    closed.close()
    for call in (lambda: arf.rotary(closed, q, None, pos, arf.RotaryTable(64)),
                 lambda: arf.paged_decode(closed, q, cache, table, pos),
                 lambda: arf.copy_pages(closed, cache, [], []),
                 lambda: arf.rotary_append(closed, None, k, k, None, pos.long(), None, cache)):
        with pytest.raises(arf.ArfError) as e:
            call()
        assert e.value.status == arf.ARF_ERR_INVALID_ARG


def test_rotary_past_32_bit_offsets(ws):
    """More than 2^31 elements; the last tokens against the formula."""
    T, H, D = 270000, 64, 128
    q = torch.empty(T, H, D, dtype=BF16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    out, _ = arf.rotary(ws, q, None, pos, arf.RotaryTable(D))
    for at in (slice(0, 2), slice(131071, 131073), slice(262143, 262145), slice(T - 3, T)):
        want, bound = ref.rotate(q[at].cpu(), pos[at].cpu(), inv_freq(D), D, False)
        ref.assert_close(out[at], want, bound + ref.half_step(want, BF16) + want.abs().amax() * 2.0 ** -30, str(at))


# ---- pages -------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, FP16, E4M3])
@pytest.mark.parametrize("form", ["nhd", "hnd", "interleaved", "heads", "rows"])
def test_copy_pages(ws, dtype, form):
    D = 64
    n, size, H = 40, 5, 3
    caches, before = [], []
    for i in range(3):
        if form == "interleaved":
            base = pages(n, 2 * size, H, D, dtype, "nhd", i).to(DEV)
            k, v = base.view(n, 2, size, H, D)[:, 0], base.view(n, 2, size, H, D)[:, 1]
        elif form == "heads":
            base = pages(n, size, 2 * H + 1, D, dtype, "nhd", i).to(DEV)
            k, v = base[:, :, :H], base[:, :, H + 1:]
        elif form == "rows":
            base = pages(n, 2 * size, H, D, dtype, "hnd", i).to(DEV)
            k, v = base[:, :, :size], base[:, :, size:]
        else:
            k, v = pages(n, size, H, D, dtype, form, i).to(DEV), pages(n, size, H, D, dtype, form, 9 + i).to(DEV)
        caches.append(arf.KVCache(k, v, "hnd" if form in ("hnd", "rows") else "nhd"))
        before.append((k.cpu(), v.cpu()))
    order = torch.randperm(n, generator=gen(2)).to(torch.int32)
    src, dst = order[:15], order[15:30]
    src[4] = src[3]           # one page to two places
    src[7] = dst[7]           # copies nothing
    arf.copy_pages(ws, caches, src, dst)
    for c, (k, v) in zip(caches, before):
        for got, want in ((c.k, k), (c.v, v)):
            want = want.view(torch.uint8) if dtype == E4M3 else want
            want = want.clone()
            want[dst.long()] = want[src.long()]
            got = got.cpu().contiguous()
            assert torch.equal((got.view(torch.uint8) if dtype == E4M3 else got), want)


def test_copy_many_pairs_and_caches(ws):
    L, n = 70, 2600  # more than one launch's pointers and pairs
    kv = torch.randint(-30000, 30000, (L, 2, n, 1, 1, 8), generator=gen(1), dtype=torch.int16).to(DEV)
    x = kv.view(FP16)
    caches = [arf.KVCache(x[i, 0], x[i, 1]) for i in range(L)]
    order = torch.randperm(n, generator=gen(2)).to(torch.int32)
    want = kv.clone()
    want[:, :, order[1300:].to(DEV).long()] = kv[:, :, order[:1300].to(DEV).long()]
    arf.copy_pages(ws, caches, order[:1300], order[1300:])
    assert torch.equal(kv, want)
    arf.copy_pages(ws, caches, [], [])
    assert torch.equal(kv, want)


def test_copy_wrapper_refuses(ws):
    k = torch.zeros(4, 16, 2, 64, dtype=BF16, device=DEV)
    cache = arf.KVCache(k, k.clone())
    for a in (([], [0], [1]), (cache, [0, 1], [2]), (cache, torch.tensor([0]), [1]),
              (cache, torch.zeros(1, dtype=torch.int32, device=DEV), [1])):
        with pytest.raises(ValueError):
            arf.copy_pages(ws, *a)
    for a in (([0, 1], [2, 2]), ([0, 1], [1, 2]), ([0], [4]), ([-1], [2])):
        with pytest.raises(arf.ArfError):
            arf.copy_pages(ws, cache, *a)
    assert not k.any()


def test_forked_sequences_through_the_pool(ws):
    """Sequences that open, fork, grow with copies of shared pages, end and
    are compacted: their tokens, read back and attended to, stay their own."""
    page, H, D, n = 4, 1, 64, 24
    kd, vd = (torch.zeros(n, page, H, D, dtype=BF16, device=DEV) for _ in range(2))
    cache = arf.KVCache(kd, vd)
    tokens = {}
    count = itertools.count(1)

    def write(pool, seq, first):
        new = pool.length(seq) - first
        k, v = randn((new, H, D), BF16, next(count)), randn((new, H, D), BF16, 1000 + next(count))
        p = torch.tensor(pool.pages(seq))
        j = torch.arange(first, first + new)
        arf.rotary_append(ws, None, k.to(DEV), v.to(DEV), None, (p[j // page] * page + j % page).to(DEV), None, cache)
        tokens.setdefault(seq, [])
        tokens[seq] = tokens[seq] + list(zip(k, v))

    def grow(pool, seq, m):
        first = pool.length(seq)
        move = pool.extend(seq, m)
        if move:
            arf.copy_pages(ws, cache, [move[0]], [move[1]])
        write(pool, seq, first)

    with arf.PagePool(n, page) as pool:
        a = pool.open(10)
        write(pool, a, 0)
        b = pool.fork(a)
        tokens[b] = list(tokens[a])
        grow(pool, b, 3)
        grow(pool, a, 1)
        c = pool.fork(b)
        tokens[c] = list(tokens[b])
        grow(pool, c, 9)
        pool.free(a)
        del tokens[a]
        d = pool.open(0)
        grow(pool, d, 5)
        pool.free(b)
        del tokens[b]
        src, dst = pool.compact()
        assert len(src) > 0
        arf.copy_pages(ws, cache, src, dst)
        seqs = [c, d]
        table, lens = pool.block_table(seqs, width=8)
    q = randn((2, 2, D), BF16, 77)
    got = arf.paged_decode(ws, q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    for i, s in enumerate(seqs):
        for j, (k, v) in enumerate(tokens[s]):
            p = int(table[i, j // page])
            assert same(kd[p, j % page], k) and same(vd[p, j % page], v)
    ref.assert_decode(got, ref.decode(q, kd.cpu(), vd.cpu(), "nhd", table, lens, D ** -0.5), BF16)


# ---- a decode step of a tensor-parallel layer ----------------------------------


@pytest.mark.parametrize("dtype,W", [(BF16, 2), (FP16, 4)])
def test_decode_step_between_two_epilogues(ws, dtype, W):
    """W shards' attention of one step, output projections, and the epilogue
    that sums their partials: against the whole layer in 64 bits."""
    B, Hkv, G, D, page, H = 5, 1, 4, 64, 16, 512
    eps = 1e-5
    parts, want, slack = [], torch.zeros(B, H, dtype=torch.float64), torch.zeros(B, H, dtype=torch.float64)
    lens = torch.tensor([40, 1, 17, 64, 33], dtype=torch.int32)
    rot = arf.RotaryTable(D, base=500000.0)
    pos = lens - 1
    for r in range(W):
        q, kp, vp, table, _ = batch(lens.tolist(), page, Hkv, G, D, dtype, dtype, "nhd", seed=100 * r, nan=False)
        k, v = randn((B, Hkv, D), dtype, 7 + r), randn((B, Hkv, D), dtype, 17 + r)
        w = randn((Hkv * G * D, H), dtype, 27 + r, (Hkv * G * D * W) ** -0.5)
        at = pos.long()
        slots = table.gather(1, (at // page)[:, None])[:, 0].long() * page + at % page
        cache = arf.KVCache(kp.to(DEV), vp.to(DEV))
        qr = arf.rotary_append(ws, q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), slots.to(DEV), rot, cache)
        out, _ = arf.paged_decode(ws, qr, cache, table.to(DEV), lens.to(DEV))
        parts.append(out.flatten(1).float() @ w.to(DEV).float())
        # 64 bits, from the stored (rounded) queries and keys
        o, _, tol, _ = ref.decode(qr.cpu(), cache.k.cpu(), cache.v.cpu(), "nhd", table, lens, D ** -0.5)
        qw, qb = ref.rotate(q, pos, inv_freq(D, 500000.0), D, False)
        ref.assert_close(qr, qw, qb + ref.half_step(qw, dtype), "queries")
        want += o.flatten(1) @ w.double()
        # out's own rounding and bound, through the projection; the float32
        # product's sums over Hkv G D terms
        slack += (tol + ref.half_step(o, dtype)).flatten(1) @ w.double().abs()
        slack += o.flatten(1).abs() @ w.double().abs() * (Hkv * G * D) * 2.0 ** -24
    residual, gamma = randn((B, H), dtype, 90), randn((H,), dtype, 91).abs() + 0.5
    gamma = gamma.to(dtype)
    y, ro = arf.run(ws, "rmsnorm", parts, residual.to(DEV), gamma.to(DEV), eps)
    full = want + residual.double()
    bound = slack + full.abs() * (W + 1) * 2.0 ** -23
    ref.assert_close(ro, full, bound + ref.half_step(full.abs() + bound, dtype), "residual_out")
    x = ro.cpu().double()
    norm = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gamma.double()
    ref.assert_close(y, norm, 2 * ref.half_step(norm * 1.01, dtype), "out")


# ---- what the launch before has written ------------------------------------------


@pytest.mark.parametrize("width", [4, 4000])
def test_replayed_append_copy_and_decode(ws, width):
    """Append, page copy and attention back to back in one graph, each reading
    what the launch before it wrote, with other data in every replay."""
    page, H, G, D, B = 8, 2, 4, 64, 4
    n = page  # one page per sequence, filled by the append and copied
    kp, vp = (torch.zeros(2 * B, page, H, D, dtype=BF16, device=DEV) for _ in range(2))
    cache = arf.KVCache(kp, vp)
    q, k, v = (torch.zeros(B * n, h, D, dtype=BF16, device=DEV) for h in (H * G, H, H))
    pos = torch.arange(B * n, dtype=torch.int32, device=DEV) % n
    slots = torch.arange(B * n, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32)
    table[:, 0] = torch.arange(B, 2 * B)
    table, lens = table.to(DEV), torch.full((B,), n, dtype=torch.int32, device=DEV)
    size = ctypes.c_size_t()
    assert arf.arf_paged_decode_scratch_bytes(ws.handle, cache.struct, B, H * G, width, 0, size) == arf.ARF_OK
    assert (size.value > 0) == (width == 4000), "both forms are meant"
    rot = arf.RotaryTable(D)

    def step():
        qr = arf.rotary_append(ws, q, k, v, pos, slots, rot, cache)
        arf.copy_pages(ws, cache, list(range(B)), list(range(B, 2 * B)))
        last = qr[n - 1::n]
        return last, arf.paged_decode(ws, last, cache, table, lens)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        last, got = step()
    for it in range(20):
        for x, seed in ((q, 1), (k, 2), (v, 3)):
            x.copy_(randn(tuple(x.shape), BF16, 10 * it + seed))
        g.replay()
        torch.cuda.synchronize()
        assert same(vp[:B].flatten(0, 1), v) and same(vp[B:], vp[:B]) and same(kp[B:], kp[:B])
        want, bound = ref.rotate(k.cpu(), pos.cpu(), inv_freq(D), D, False)
        ref.assert_close(kp[B:].flatten(0, 1), want, bound + ref.half_step(want, BF16))
        ref.assert_decode(got, ref.decode(last.cpu(), kp.cpu(), vp.cpu(), "nhd", table[:, :1].cpu(), lens.cpu(),
                                          D ** -0.5), BF16, f"replay {it}")


def test_clusters_join_what_arrives(ws):
    """Clusters of every size, many times over with other data: the first CTA
    of each reads what the others sent, not what was there before."""
    D, Hkv, G = 128, 1, 4
    for tokens in (100, 200, 500, 1000):
        cases = [batch([tokens, tokens - 7], 16, Hkv, G, D, BF16, BF16, "nhd", seed=s) for s in range(4)]
        size = ctypes.c_size_t()
        held = []
        for q, kp, vp, table, n in cases:
            cache = arf.KVCache(kp.to(DEV), vp.to(DEV))
            st = arf.arf_paged_decode_scratch_bytes(ws.handle, cache.struct, 2, G, table.shape[1], 0, size)
            assert (st, size.value) == (arf.ARF_OK, 0), "the cluster form is meant"
            held.append((q.to(DEV), cache, table.to(DEV), n.to(DEV)))
        got = [[arf.paged_decode(ws, *a) for a in held] for _ in range(50)]
        for i, (q, kp, vp, table, n) in enumerate(cases):
            ref.assert_decode(got[0][i], ref.decode(q, kp, vp, "nhd", table, n, D ** -0.5), BF16, f"{tokens}")
            for again in got[1:]:
                assert same(again[i][0], got[0][i][0]) and same(again[i][1], got[0][i][1])
    assert wait_timeouts(ws) == 0


def wait_timeouts(ws):
    n = ctypes.c_uint()
    assert arf.arf_workspace_wait_timeouts(ws.handle, n) == arf.ARF_OK
    return n.value


def pool_stream(t):
    """The stream in whose pool of the caching allocator a tensor lies."""
    at = t.untyped_storage().data_ptr()
    return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"]][0]


def test_outputs_on_another_stream_lie_in_its_memory(ws):
    q, k = (randn((5, h, 64), BF16, h).to(DEV) for h in (4, 2))
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    cache = arf.KVCache(*(torch.zeros(4, 16, 2, 64, dtype=BF16, device=DEV) for _ in range(2)))
    table, lens = torch.zeros(5, 1, dtype=torch.int32, device=DEV), pos + 1
    rot = arf.RotaryTable(64)
    torch.cuda.synchronize()
    here, s = torch.cuda.current_stream(), torch.cuda.Stream()
    for stream, where in ((None, here), (here, here), (s, s)):
        made = [*arf.rotary(ws, q, k, pos, rot, stream=stream), arf.rotary(ws, q, None, pos, rot, stream=stream)[0],
                arf.rotary_append(ws, q, k, k, pos, pos.long(), rot, cache, stream=stream)]
        if stream is s:
            s.synchronize()
        made += arf.paged_decode(ws, q, cache, table, lens, stream=stream)
        made += [arf.paged_decode(ws, q, cache, table, lens, lse=made[-1], stream=stream)[0]]
        assert {pool_stream(x) for x in made} == {where.cuda_stream}
        torch.cuda.synchronize()


def test_memory_in_use_elsewhere_is_not_written(ws):
    """A call on another stream while work queued on the current one still
    reads tensors that were freed: neither its outputs nor its scratch are
    theirs."""
    Hkv, G, D, B = 1, 4, 64, 4
    q, kp, vp, table, n = batch([5000, 17, 0, 300], 16, Hkv, G, D, BF16, BF16, "nhd", width=4000)
    want = ref.decode(q, kp, vp, "nhd", table[:, :320], n, D ** -0.5)
    cache = arf.KVCache(kp.to(DEV), vp.to(DEV))
    q, table, n = q.to(DEV), table.to(DEV), n.to(DEV)
    size = ctypes.c_size_t()
    assert arf.arf_paged_decode_scratch_bytes(ws.handle, cache.struct, B, Hkv * G, table.shape[1], 0, size) == arf.ARF_OK
    assert size.value > 0, "the form with scratch is meant"
    s = torch.cuda.Stream()
    for warm in range(3):  # modules loaded, pools filled
        arf.paged_decode(ws, q, cache, table, n, stream=s)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sizes = [size.value, B * Hkv * G * D * 2 + 256, B * Hkv * G * D * 2 + B * Hkv * G * 4, 1 << 20]
    kept = [torch.empty(x, dtype=torch.uint8, device=DEV) for x in sizes]
    temps = [torch.full((x,), 91, dtype=torch.uint8, device=DEV) for x in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    for x, y in zip(temps, kept):
        y.copy_(x)
    freed = {x.data_ptr() for x in temps}
    del temps, x
    got = [arf.paged_decode(ws, q, cache, table, n, stream=s) for _ in range(8)]
    busy = not torch.cuda.current_stream().query()
    here = [torch.empty(x, dtype=torch.uint8, device=DEV) for x in sizes for _ in range(4)]
    again = [x.data_ptr() for x in here]
    torch.cuda.synchronize()
    assert busy, "the calls were made after the work on the current stream had ended"
    assert freed & set(again), "nothing that was freed could have been handed out"
    for y in kept:
        assert bool((y == 91).all())
    for g in got:
        ref.assert_decode(g, want, BF16)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_decode_infinite_queries_on_an_e4m3_cache(ws, dtype):
    """A query with an infinity beside large finite values: scores of -inf are
    masked out, and the finite values do not turn them into NaN."""
    D, n, large = 64, 40, 1e30 if dtype == BF16 else 6e4
    q = torch.zeros(1, 3, D, dtype=dtype)
    q[..., 1], q[..., 2] = large, -large
    q[0, 0, 0] = -math.inf    # every score is -inf
    q[0, 1, 0] = math.inf     # +inf: the whole row is NaN
    g = gen(3)
    k = torch.zeros(3, 16, 1, D)
    k[..., 0] = 1.0
    k[..., 1:] = torch.randint(1, 5, (3, 16, 1, D - 1), generator=g).float()
    v = torch.randn(3, 16, 1, D, generator=g)
    kd, vd = k.to(E4M3), v.to(E4M3)
    table, lens = torch.arange(3, dtype=torch.int32)[None], torch.tensor([n], dtype=torch.int32)
    args = (table.to(DEV), lens.to(DEV))
    out, lse = (x.cpu() for x in arf.paged_decode(ws, q.to(DEV), arf.KVCache(kd.to(DEV), vd.to(DEV)), *args,
                                                  scale=1.0 / large))
    assert not out[0, 0].any() and lse[0, 0] == -math.inf
    assert bool(out[0, 1].isnan().all())
    q[0, :2] = q[0, 2]
    want = ref.decode(q, kd, vd, "nhd", table, lens, 1.0 / large)
    ref.assert_close(out[0, 2], want[0][0, 2], want[2][0, 2] + ref.half_step(want[0][0, 2], dtype))
    ref.assert_close(lse[0, 2], want[1][0, 2], want[3][0, 2])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("width", [1, 4000])
def test_decode_probabilities_on_an_e4m3_cache(ws, D, width):
    """Values whose weighted sum cancels: what is left shows the rounding of
    the probabilities, which out's own does not hide. They enter the product
    as two fp16 values, off by 2^-16 of sum p |v| / sum p, for bf16 queries
    too. Small queries keep the bound on the scores' own error below that."""
    B, n, page = 64, 2, 16
    g = gen(D)
    q = (torch.randn(B, 1, D, generator=g) / D).to(BF16)
    k = torch.randn(B, page, 1, D, generator=g).to(E4M3)
    v = torch.empty(B, page, 1, D)
    table = torch.full((B, width), -1, dtype=torch.int32)
    table[:, 0] = torch.arange(B)
    lens = torch.full((B,), n, dtype=torch.int32)
    # both weights are near a half: the values +1, -1 leave their difference
    v[:, 0::2], v[:, 1::2] = 1.0, -1.0
    v = v.to(E4M3)
    got = arf.paged_decode(ws, q.to(DEV), arf.KVCache(k.to(DEV), v.to(DEV)), table.to(DEV), lens.to(DEV))
    out, lse, tol, ltol = ref.decode(q, k, v, "nhd", table[:, :1], lens, D ** -0.5)
    # sum p |v| / sum p is 1 here; ref's bound holds 2^-11 of it
    ref.assert_close(got[0], out, tol - 2.0 ** -11 + 2.0 ** -16 + ref.half_step(out, BF16), "out")
    ref.assert_close(got[1], lse, ltol, "lse")


def test_decode_more_heads_than_32_bits_of_chunks(ws):
    """Heads times their 8-byte chunks beyond 2^31: a sequence without tokens
    is answered in every head, one with a token too."""
    D, heads, page = 256, (1 << 25) + 8, 16
    kp, vp = (torch.randn(1, page, 1, D, generator=gen(i)).to(BF16).to(DEV) for i in (1, 2))
    q = torch.ones(1, 1, D, dtype=BF16, device=DEV).expand(-1, heads, -1)
    out = torch.full((1, heads, D), 3.0, dtype=BF16, device=DEV)
    lse = torch.zeros(1, heads, device=DEV)
    table = torch.zeros(1, 40, dtype=torch.int32, device=DEV)
    cache, size = arf.KVCache(kp, vp), ctypes.c_size_t()
    assert arf.arf_paged_decode_scratch_bytes(ws.handle, cache.struct, 1, heads, 40, 0, size) == arf.ARF_OK
    assert size.value > 0, "the dealt form is meant"
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    arf.paged_decode(ws, q, cache, table, lens, out=out, lse=lse)
    assert bool((lse == -math.inf).all()) and not out.any()
    arf.paged_decode(ws, q, cache, table, lens + 1, out=out, lse=lse)
    assert bool((out == vp[0, 0]).all()) and bool((lse == lse[0, 0]).all())


# ---- autograd --------------------------------------------------------------------


def test_gradients_are_refused(ws):
    q, k = (randn((2, h, 64), BF16, h).to(DEV) for h in (4, 2))
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    kp, vp = (torch.zeros(2, 16, 2, 64, dtype=BF16, device=DEV) for _ in range(2))
    cache, rot, table = arf.KVCache(kp, vp), arf.RotaryTable(64), pos[:, None].contiguous()
    grad = lambda x: x.clone().requires_grad_()  # noqa: E731
    lse = torch.zeros(2, 4, device=DEV)
    calls = [lambda: arf.rotary(ws, grad(q), k, pos, rot), lambda: arf.rotary(ws, q, grad(k), pos, rot),
             lambda: arf.rotary(ws, q, k, pos, rot, q_out=grad(q)), lambda: arf.rotary(ws, q * grad(q), None, pos, rot),
             lambda: arf.rotary_append(ws, q, k, grad(k), pos, pos.long(), rot, cache),
             lambda: arf.rotary_append(ws, q, grad(k), k, pos, pos.long(), rot, cache),
             lambda: arf.paged_decode(ws, grad(q), cache, table, pos), lambda: arf.paged_decode(ws, q, cache, table, pos, lse=grad(lse)),
             lambda: arf.paged_decode(ws, q, cache, table, pos, out=grad(q))]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            for call in calls:
                call()
    for pages_ in ((kp, grad(vp)), (grad(kp), vp), (grad(kp)[:1], vp[:1])):
        with pytest.raises(ValueError, match="gradient"):
            arf.KVCache(*pages_)


def test_what_a_call_writes_counts_as_modified(ws):
    """Autograd must not use what it saved of a tensor that a call has
    overwritten."""
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    rot = arf.RotaryTable(64)

    def stale(x, call):
        w = torch.ones((), dtype=x.dtype, device=DEV, requires_grad=True)
        y = (w * x).sum()  # saves x
        version = x._version
        call()
        assert x._version > version
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()

    q, k = (randn((2, h, 64), BF16, h).to(DEV) for h in (4, 2))
    stale(q, lambda: arf.rotary(ws, q, None, pos, rot, q_out=q))
    stale(k, lambda: arf.rotary(ws, q, k, pos, rot, k_out=k))
    for i in range(2):
        pages_ = [torch.zeros(2, 16, 2, 64, dtype=BF16, device=DEV) for _ in range(2)]
        cache = arf.KVCache(*pages_)
        stale(pages_[i], lambda: arf.rotary_append(ws, None, k, k, None, pos.long(), None, cache))
        stale(pages_[i], lambda: arf.copy_pages(ws, [cache], [0], [1]))
        # views of one tensor, separate tensors and other views of both, in one call
        both, views = torch.zeros(2, 2, 2, 16, 2, 64, dtype=BF16, device=DEV), pages_[i].detach()
        many = [arf.KVCache(both[0, 0], both[0, 1]), cache, arf.KVCache(both[1, 0], both[1, 1])]
        stale(both, lambda: arf.copy_pages(ws, many, [0], [1]))
        stale(pages_[i], lambda: arf.copy_pages(ws, many, [0], [1]))
        stale(pages_[i], lambda: arf.copy_pages(ws, arf.KVCache(views, torch.zeros_like(views)), [0], [1]))
    out, lse = torch.zeros_like(q), torch.zeros(2, 4, device=DEV)
    stale(out, lambda: arf.paged_decode(ws, q, cache, pos[:, None], pos, out=out))
    stale(lse, lambda: arf.paged_decode(ws, q, cache, pos[:, None], pos, lse=lse))
    stale(out, lambda: arf.rotary_append(ws, q, k, k, pos, pos.long(), rot, cache, q_out=out))
    with torch.inference_mode():  # has no versions
        x = torch.zeros_like(q)
        arf.rotary(ws, q, None, pos, rot, q_out=x)


def test_keys_and_values_that_share_elements(ws):
    """They can be read, not written; views that only interleave can."""
    page, H, D = 8, 2, 64
    base = torch.randn(6, 2 * page, H, D, generator=gen(1)).to(BF16).to(DEV)
    before = base.clone()
    k = randn((3, H, D), BF16, 2).to(DEV)
    slots = torch.arange(3, device=DEV)
    q, table, lens = randn((1, 4, D), BF16, 3).to(DEV), torch.arange(3, dtype=torch.int32)[None], torch.tensor([20])
    for a, b in ((base[:4, :page], base[:4, :page]), (base[:4, :page], base[1:5, :page]),
                 (base[:4, :page], base[:4, 1:page + 1]), (base[:4, :page], base[1:5, page - 1:2 * page - 1])):
        cache = arf.KVCache(a, b)
        for call in (lambda: arf.rotary_append(ws, None, k, k, None, slots, None, cache),
                     lambda: arf.copy_pages(ws, cache, [0], [1])):
            with pytest.raises(ValueError, match="share"):
                call()
        got = arf.paged_decode(ws, q, cache, table.to(DEV), lens.int().to(DEV))
        want = ref.decode(q.cpu(), a.cpu(), b.cpu(), "nhd", table, lens, D ** -0.5)
        ref.assert_decode(got, want, BF16)
    assert torch.equal(base, before)
    cache = arf.KVCache(base[:, :page], base[:, page:])
    arf.rotary_append(ws, None, k, k, None, slots, None, cache)
    arf.copy_pages(ws, cache, [0], [1])
    assert torch.equal(base[1], base[0]) and torch.equal(base[0, :3], k) and torch.equal(base[0, page:page + 3], k)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_given_frequencies(ws, interleaved):
    """Frequencies that no named scaling has: a ramp linear in the pair's
    index between the pairs of 32 turns and of 1 turn, its factor given."""
    rot, D, base, factor, length = 64, 80, 10000.0, 16.0, 4096
    w = inv_freq(rot, base)
    at = lambda turns: rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = math.floor(at(32.0)), math.ceil(at(1.0))
    keep = 1.0 - ((torch.arange(rot // 2, dtype=torch.float64) - lo) / (hi - lo)).clamp(0, 1)
    w = w * (keep + (1.0 - keep) / factor)
    pos = torch.randint(0, 60000, (50,), generator=gen(1), dtype=torch.int32)
    q = randn((50, 3, D), BF16, 2)
    for magnitude in (1.0, 0.1 * math.log(factor) + 1.0):
        table = arf.RotaryTable.from_frequencies(w, magnitude, "interleaved" if interleaved else "half")
        qo, _ = arf.rotary(ws, q.to(DEV), None, pos.to(DEV), table)
        want, bound = ref.rotate(q, pos, w, rot, interleaved, magnitude)
        ref.assert_close(qo, want, bound + ref.half_step(want, BF16))
        assert same(qo[..., rot:], q[..., rot:])


# ---- the form with scratch, on several streams, threads and graphs ------------------


def wide_batch(ws, lens, seed, Hkv=1, G=4, D=64, width=4000):
    """A batch whose table is wide enough for the dealt form: (arguments of
    paged_decode on the device, the expected result)."""
    q, kp, vp, table, n = batch(lens, 16, Hkv, G, D, BF16, BF16, "nhd", seed=seed, width=width)
    cache, size = arf.KVCache(kp.to(DEV), vp.to(DEV)), ctypes.c_size_t()
    assert arf.arf_paged_decode_scratch_bytes(ws.handle, cache.struct, len(lens), Hkv * G, width, 0, size) == arf.ARF_OK
    assert size.value > 0, "the form with scratch is meant"
    return (q.to(DEV), cache, table.to(DEV), n.to(DEV)), ref.decode(q, kp, vp, "nhd", table, n, D ** -0.5)


def test_decode_with_scratch_on_several_streams(ws):
    cases = [wide_batch(ws, [5000, 17, 0, 300 + i], 10 * i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(30):
        got = [arf.paged_decode(ws, *args, stream=s) for s, (args, _) in zip(streams, cases)]
    torch.cuda.synchronize()
    for g, (_, want) in zip(got, cases):
        ref.assert_decode(g, want, BF16)


def test_decode_with_scratch_from_two_threads(ws):
    import threading
    cases, errors = [wide_batch(ws, [9000, 17, 0, 300 + i], 10 * i) for i in range(2)], []
    torch.cuda.synchronize()

    def work(args, want):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got = [arf.paged_decode(ws, *args) for _ in range(50)]
                s.synchronize()
            for g in got[::7]:
                ref.assert_decode(g, want, BF16)
        except Exception as e:  # noqa: BLE001  (reported by the test's thread)
            errors.append(e)
    ts = [threading.Thread(target=work, args=c) for c in cases]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not errors, errors


def test_graphs_with_scratch_share_a_workspace(ws):
    """Two graphs captured with one workspace, replayed at the same time."""
    cases = [wide_batch(ws, [9000, 17, 0, 4000 + i], 10 * i) for i in range(2)]
    streams, graphs, outs = [torch.cuda.Stream() for _ in cases], [], []
    for s, (args, _) in zip(streams, cases):
        arf.paged_decode(ws, *args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(arf.paged_decode(ws, *args))
        graphs.append(g)
    for it in range(10):
        for o in outs:
            o[0].fill_(5.0)
        torch.cuda.synchronize()
        for _ in range(20):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for o, (_, want) in zip(outs, cases):
            ref.assert_decode(o, want, BF16, f"replay {it}")


def check_before_window(ws, lens, page, D, cdt, layout, window, scratch):
    """NaN in every row before the window, and no page at all (-1) where a
    page lies wholly before it: neither is read, neither is counted."""
    ks = 0.02 if cdt == E4M3 else 1.0
    q, kp, vp, table, n = batch(lens, page, 1, 3, D, BF16, cdt, layout, seed=window, ks=ks, vs=ks)
    want = ref.decode(q, kp, vp, layout, table, n, D ** -0.5, 0.0, window, ks, ks)
    slot = torch.arange(table.shape[1] * page)
    for p in (kp, vp):
        x = p.view(torch.uint8) if cdt == E4M3 else p
        x = x if layout == "nhd" else x.transpose(1, 2)
        for b, m in enumerate(lens):
            j = slot[: max(0, m - window)]
            x[table[b, j // page].long(), j % page] = 0x7F if cdt == E4M3 else math.nan
    for b, m in enumerate(lens):
        table[b, : max(0, m - window) // page] = -1
    cache, size = arf.KVCache(kp.to(DEV), vp.to(DEV), layout, ks, ks), ctypes.c_size_t()
    assert arf.arf_paged_decode_scratch_bytes(ws.handle, cache.struct, len(lens), 3, table.shape[1], window,
                                              size) == arf.ARF_OK and (size.value > 0) == scratch
    got = arf.paged_decode(ws, q.to(DEV), cache, table.to(DEV), n.to(DEV), window=window)
    ref.assert_decode(got, want, BF16, f"{page} {window} {D}")
    assert arf.bad_indices(ws) == 0


@pytest.mark.parametrize("page", [16, 5, 64])
@pytest.mark.parametrize("window", [1, 15, 33, 100])
def test_decode_reads_nothing_before_the_window(ws, page, window):
    for D, cdt, layout in ((64, BF16, "nhd"), (128, E4M3, "hnd"), (256, BF16, "nhd")):
        check_before_window(ws, [300, 33, 1, 64, window, window + 1, 0], page, D, cdt, layout, window, False)


@pytest.mark.parametrize("page", [16, 5, 64])
def test_decode_with_scratch_reads_nothing_before_the_window(ws, page):
    check_before_window(ws, [40011, 20000, 0, 20001, 20077], page, 64, BF16, "nhd", 20000, True)
    check_before_window(ws, [40011, 20000, 0, 20001, 20077], page, 128, E4M3, "hnd", 20000, True)
