"""The attention operators on the host (no GPU): rotary tables against the
formulas, refusals of the C entry points and of the Python wrappers, and the
page pool against a model of it."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

import all_reduce_residual_gb300 as arf
from all_reduce_residual_gb300 import build

INVALID, UNSUPPORTED = arf.ARF_ERR_INVALID_ARG, arf.ARF_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    arf.load()


@pytest.fixture()
def no_ws():
    """Memory that passes for a workspace of no device: a call whose arguments
    are in order ends at the device check, with an error and no launch."""
    buf = (ctypes.c_uint8 * 8192)()
    ctypes.memset(buf, 0xFF, 8192)
    return ctypes.c_void_p(ctypes.addressof(buf)), buf


def stopped_at_device(st):
    return st in (arf.ARF_ERR_CUDA, arf.ARF_ERR_DEVICE_MISMATCH)


# ---- rotary tables -----------------------------------------------------------


def turns(rot, base=10000.0, scaling=arf.ARF_ROPE_NONE, factor=1.0, length=4096.0, fast=32.0, slow=1.0):
    out, mag = (ctypes.c_uint64 * max(1, rot // 2))(), ctypes.c_float(-1.0)
    return arf.arf_rotary_turns(rot, base, scaling, factor, length, fast, slow, out, mag), list(out), mag.value


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [("NONE", 1.0), ("LINEAR", 8.0), ("NTK", 4.0), ("YARN", 16.0),
                                            ("YARN", 1.0)])
def test_rotary_turns_follow_the_formulas(rot, scaling, factor):
    if scaling == "NTK" and rot == 2:
        pytest.skip("refused: rot / (rot - 2)")
    st, got, mag = turns(rot, 500000.0, getattr(arf, "ARF_ROPE_" + scaling), factor, 8192.0)
    assert st == arf.ARF_OK
    for i in range(rot // 2):
        base = 500000.0 * factor ** (rot / (rot - 2)) if scaling == "NTK" else 500000.0
        w = base ** (-2.0 * i / rot)
        if scaling == "LINEAR":
            w /= factor
        if scaling == "YARN":
            r = 8192.0 * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (r - 1.0) / 31.0))
            w *= keep + (1.0 - keep) / factor
        want = w / (2 * math.pi) * 2.0 ** 64
        # power, logarithm and a few products in binary64, each off by an ulp
        # or so, the power's exponent by its own relative error
        assert abs(got[i] - want) <= want * 2.0 ** -46 + 1
    want_mag = 0.1 * math.log(factor) + 1 if scaling == "YARN" else 1.0
    assert abs(mag - want_mag) <= want_mag * 2.0 ** -24


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=3), dict(rot=-2), dict(rot=8, base=1.0),
                                dict(rot=8, base=math.inf), dict(rot=8, factor=0.5), dict(rot=8, factor=math.nan),
                                dict(rot=2, scaling=arf.ARF_ROPE_NTK, factor=2.0),
                                dict(rot=8, scaling=arf.ARF_ROPE_YARN, fast=1.0, slow=1.0),
                                dict(rot=8, scaling=arf.ARF_ROPE_YARN, length=0.0),
                                dict(rot=8, scaling=arf.ARF_ROPE_YARN, slow=-math.inf), dict(rot=8, scaling=7)])
def test_rotary_turns_refuse(kw):
    assert turns(**kw)[0] == INVALID


def test_rotary_table_refuses_unknown_names():
    with pytest.raises(ValueError):
        arf.RotaryTable(8, layout="neighbours", device="cpu")
    with pytest.raises(ValueError):
        arf.RotaryTable(8, scaling="other", device="cpu")
    with pytest.raises(arf.ArfError):
        arf.RotaryTable(7, device="cpu")
    t = arf.RotaryTable(8, device="cpu")
    assert t.turns.shape == (4,) and t.struct.interleaved == 0
    # position times turns modulo 2^64: whole turns drop out exactly
    f = [x % (1 << 64) for x in t.turns.tolist()]
    for pos in (1, 4097, 2 ** 31 - 1):
        for i, x in enumerate(f):
            frac = (x * pos % (1 << 64)) / 2.0 ** 64
            exact = math.fmod(pos * 10000.0 ** (-2 * i / 8) / (2 * math.pi), 1.0)
            assert min(abs(frac - exact), 1 - abs(frac - exact)) <= pos * 2.0 ** -52


# ---- refusals of the C entry points --------------------------------------------

FAR = 1 << 20  # an address no call here follows


def heads(data=FAR, ts=1024, hs=128, n=8):
    return arf.Heads(data, ts, hs, n)


def cache(**kw):
    f = dict(k=FAR, v=FAR, num_pages=10, page_size=16, kv_heads=2, head_dim=128, page_stride=4096, token_stride=256,
             head_stride=128, dtype=arf.ARF_BF16, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return arf.Cache(**f)


def rot(**kw):
    f = dict(turns=FAR, rot_dim=128, interleaved=0, magnitude=1.0)
    f.update(kw)
    return arf.Rotary(**f)


def call_rotary(ws, **kw):
    a = dict(rot=rot(), positions=FAR, T=3, D=128, dtype=arf.ARF_BF16, q=heads(), q_out=heads(2 * FAR), k=heads(n=2),
             k_out=heads(3 * FAR, n=2), stream=0)
    a.update(kw)
    return arf.arf_rotary(ws, *a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rot=None), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(dtype=2), INVALID),
    (dict(rot=rot(rot_dim=130)), INVALID), (dict(rot=rot(rot_dim=3)), INVALID), (dict(rot=rot(rot_dim=0)), INVALID),
    (dict(rot=rot(magnitude=math.nan)), INVALID), (dict(rot=rot(turns=None)), INVALID),
    (dict(rot=rot(turns=FAR + 4)), UNSUPPORTED), (dict(positions=None), INVALID), (dict(positions=FAR + 2), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(q=heads(data=None)), INVALID),
    (dict(q=heads(n=0)), INVALID), (dict(q=heads(n=7)), INVALID), (dict(q=heads(ts=-1)), INVALID),
    (dict(q=heads(data=FAR + 1)), UNSUPPORTED), (dict(k=None), INVALID), (dict(k_out=None), INVALID),
    (dict(k_out=heads(n=3)), INVALID), (dict(q_out=heads(2 * FAR, hs=64)), INVALID),
    (dict(q_out=heads(2 * FAR, ts=100)), INVALID), (dict(q=heads(ts=2048), q_out=heads()), INVALID),
    (dict(q_out=heads(2 * FAR, ts=1 << 40)), UNSUPPORTED), (dict(T=(1 << 40) + 1), UNSUPPORTED),
    (dict(D=(1 << 20) + 2), UNSUPPORTED),
])
def test_rotary_refuses(no_ws, kw, want):
    assert call_rotary(no_ws[0], **kw) == want


def test_rotary_accepts(no_ws):
    for kw in (dict(), dict(k=None, k_out=None), dict(q_out=heads()), dict(T=0), dict(D=128, rot=rot(rot_dim=6)),
               dict(q_out=heads(2 * FAR, ts=128, hs=3 * 128)), dict(T=1, q_out=heads(2 * FAR, ts=0))):
        assert stopped_at_device(call_rotary(no_ws[0], **kw)), kw
    assert call_rotary(None) == INVALID


def call_append(ws, **kw):
    a = dict(rot=rot(), positions=FAR, slots=FAR, T=3, dtype=arf.ARF_BF16, q=heads(), q_out=heads(2 * FAR),
             k=heads(n=2), v=heads(n=2), cache=cache(), stream=0)
    a.update(kw)
    return arf.arf_rotary_append(ws, *a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rot=None), INVALID), (dict(slots=None), INVALID), (dict(slots=FAR + 4), UNSUPPORTED),
    (dict(positions=None), INVALID), (dict(T=-1), INVALID), (dict(dtype=2), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=heads(n=3)), INVALID),
    (dict(v=heads(n=8)), INVALID), (dict(cache=None), INVALID), (dict(cache=cache(page_size=0)), INVALID),
    (dict(cache=cache(k=None)), INVALID), (dict(cache=cache(k_scale=0.5)), INVALID),
    (dict(cache=cache(dtype=arf.ARF_E4M3, k_scale=0.0)), INVALID),
    (dict(cache=cache(dtype=arf.ARF_E4M3, v_scale=1e-40)), INVALID),
    (dict(cache=cache(dtype=arf.ARF_E4M3, v_scale=math.inf)), INVALID), (dict(cache=cache(dtype=5)), INVALID),
    (dict(cache=cache(page_stride=-1)), INVALID), (dict(cache=cache(dtype=arf.ARF_FP16)), UNSUPPORTED),
    (dict(cache=cache(page_stride=1 << 40)), UNSUPPORTED), (dict(cache=cache(v=FAR + 1)), UNSUPPORTED),
    (dict(rot=rot(rot_dim=256)), INVALID), (dict(cache=cache(head_stride=64)), INVALID),
    (dict(cache=cache(head_stride=0)), INVALID), (dict(cache=cache(token_stride=128, head_stride=128)), INVALID),
    (dict(cache=cache(page_stride=2048)), INVALID),
])
def test_append_refuses(no_ws, kw, want):
    assert call_append(no_ws[0], **kw) == want


def test_append_accepts(no_ws):
    for kw in (dict(), dict(q=None, q_out=None), dict(rot=None, q=None, q_out=None, positions=None),
               dict(cache=cache(dtype=arf.ARF_E4M3, k_scale=0.1)), dict(q_out=heads()),
               dict(cache=cache(token_stride=128, head_stride=16 * 128)),
               dict(cache=cache(page_stride=128, token_stride=1280, head_stride=20480)),
               dict(cache=cache(num_pages=1, page_stride=0))):
        assert stopped_at_device(call_append(no_ws[0], **kw)), kw


def call_decode(ws, **kw):
    a = dict(cache=cache(), B=3, dtype=arf.ARF_BF16, q=heads(), table=FAR, ts=4, tw=4, lens=FAR, scale=0.1, cap=0.0,
             window=0, out=heads(2 * FAR), lse=FAR, scratch=FAR, nbytes=1 << 40, stream=0)
    a.update(kw)
    return arf.arf_paged_decode(ws, *a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(cache=None), INVALID), (dict(B=-1), INVALID), (dict(dtype=2), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(q=heads(n=7), out=heads(n=7)), INVALID), (dict(out=heads(n=4)), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(ts=-1), INVALID),
    (dict(tw=-1), INVALID), (dict(scale=math.nan), INVALID), (dict(cap=-1.0), INVALID), (dict(cap=math.inf), INVALID), (dict(cap=3e38), INVALID),
    (dict(cap=1e-40), INVALID), (dict(scale=3e38), INVALID),
    (dict(window=-1), INVALID), (dict(out=heads(2 * FAR, ts=64)), INVALID),
    (dict(cache=cache(head_dim=96)), UNSUPPORTED), (dict(cache=cache(dtype=arf.ARF_FP16)), UNSUPPORTED),
    (dict(cache=cache(token_stride=260)), UNSUPPORTED), (dict(cache=cache(k=FAR + 8)), UNSUPPORTED),
    (dict(cache=cache(dtype=arf.ARF_E4M3, head_stride=136)), UNSUPPORTED), (dict(q=heads(ts=1028)), UNSUPPORTED),
    (dict(q=heads(data=FAR + 2)), UNSUPPORTED), (dict(scratch=FAR + 16), UNSUPPORTED), (dict(lse=FAR + 2), UNSUPPORTED),
    (dict(lens=FAR + 2), UNSUPPORTED), (dict(B=1 << 31), UNSUPPORTED),
])
def test_decode_refuses(no_ws, kw, want):
    assert call_decode(no_ws[0], **kw) == want


def test_decode_accepts(no_ws):
    for kw in (dict(), dict(lse=None), dict(B=0, scratch=None, lens=None), dict(tw=0, ts=0, table=None),
               dict(cap=30.0, window=5), dict(cache=cache(dtype=arf.ARF_E4M3, k_scale=2.0)), dict(B=1, ts=0)):
        assert stopped_at_device(call_decode(no_ws[0], **kw)), kw


def call_copy(ws, src=(1, 2), dst=(3, 4), caches=None, n=None):
    caches = [cache()] if caches is None else caches
    s, d = (ctypes.c_int32 * max(1, len(src)))(*src), (ctypes.c_int32 * max(1, len(dst)))(*dst)
    return arf.arf_copy_pages(ws, (arf.Cache * max(1, len(caches)))(*caches), len(caches), s, d,
                              len(src) if n is None else n, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(src=(1, 2), dst=(3, 3)), INVALID), (dict(src=(1, 3), dst=(3, 4)), INVALID),
    (dict(src=(-1, 2)), INVALID), (dict(src=(1, 10)), INVALID), (dict(dst=(3, -4)), INVALID),
    (dict(dst=(10, 4)), INVALID), (dict(src=(3, 3), dst=(3, 4)), INVALID), (dict(n=-1), INVALID),
    (dict(caches=[]), INVALID), (dict(caches=[cache(), cache(page_size=8)]), INVALID),
    (dict(caches=[cache(), cache(dtype=arf.ARF_FP16)]), INVALID), (dict(caches=[cache(k=None)]), INVALID),
    (dict(caches=[cache(head_dim=100)]), UNSUPPORTED), (dict(caches=[cache(page_stride=4100)]), UNSUPPORTED),
    (dict(caches=[cache(v=FAR + 8)]), UNSUPPORTED), (dict(caches=[cache(head_stride=0)]), INVALID),
    (dict(caches=[cache(page_stride=4080)]), INVALID),
])
def test_copy_refuses(no_ws, kw, want):
    assert call_copy(no_ws[0], **kw) == want


def test_copy_accepts(no_ws):
    for kw in (dict(), dict(src=(), dst=()), dict(src=(5, 1, 1), dst=(5, 2, 3)),
               dict(caches=[cache(), cache(k=2 * FAR, k_scale=1.0)]), dict(src=(1, 1), dst=(2, 3))):
        assert stopped_at_device(call_copy(no_ws[0], **kw)), kw


def test_null_workspace_is_refused():
    assert call_append(None) == call_decode(None) == call_copy(None) == INVALID
    assert arf.arf_paged_decode_scratch_bytes(None, cache(), 3, 8, 4, 0, ctypes.c_size_t()) == INVALID
    assert arf.arf_workspace_bad_indices(None, ctypes.c_uint()) == INVALID


# ---- refusals of the Python wrappers -------------------------------------------


def test_cache_refuses():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    for kw in (dict(k=k, v=k), dict(k=k, v=k[:3]), dict(k=k.float(), v=k.float()), dict(k=k, v=k, layout="dhn"),
               dict(k=k, v=k.transpose(1, 2)), dict(k=k[0], v=k[0])):
        with pytest.raises(ValueError):
            arf.KVCache(**kw)


# ---- the page pool -------------------------------------------------------------


class Model:
    """The pool as sets and lists."""

    def __init__(self, n, size):
        self.n, self.size, self.seqs = n, size, {}

    def used(self):
        return {p for pages, _ in self.seqs.values() for p in pages}

    def free(self):
        return sorted(set(range(self.n)) - self.used())

    def holders(self, page):
        return sum(page in pages for pages, _ in self.seqs.values())


@pytest.mark.parametrize("seed", range(6))
def test_pool_follows_the_model(seed):
    rng = random.Random(seed)
    n, size = rng.choice([(1, 1), (7, 4), (40, 16), (64, 1)])
    model = Model(n, size)
    with arf.PagePool(n, size) as pool:
        for _ in range(600):
            op = rng.choice(["open", "extend", "extend", "extend", "fork", "free", "compact"])
            free = model.free()
            some = rng.choice(list(model.seqs)) if model.seqs else None
            if op == "open":
                t = rng.choice([0, 1, size, rng.randint(0, 3 * size)])
                need = -(-t // size)
                if need > len(free):
                    with pytest.raises(arf.ArfError) as e:
                        pool.open(t)
                    assert e.value.status == arf.ARF_ERR_NO_PAGES
                else:
                    s = pool.open(t)
                    assert s not in model.seqs
                    model.seqs[s] = (free[:need], t)
            elif some is None:
                continue
            elif op == "extend":
                pages, t = model.seqs[some]
                add = rng.choice([0, 1, 1, size, rng.randint(0, 2 * size)])
                copy = add > 0 and t % size != 0 and model.holders(pages[-1]) > 1
                more = -(-(t + add) // size) - len(pages)
                if more + copy > len(free):
                    with pytest.raises(arf.ArfError) as e:
                        pool.extend(some, add)
                    assert e.value.status == arf.ARF_ERR_NO_PAGES
                else:
                    got = pool.extend(some, add)
                    assert got == ((pages[-1], free[0]) if copy else None)
                    pages = pages[:-1] + free[:1] if copy else list(pages)
                    model.seqs[some] = (pages + free[int(copy):int(copy) + more], t + add)
            elif op == "fork":
                s = pool.fork(some)
                assert s not in model.seqs
                model.seqs[s] = (list(model.seqs[some][0]), model.seqs[some][1])
            elif op == "free":
                pool.free(some)
                del model.seqs[some]
            else:
                src, dst = (x.tolist() for x in pool.compact())
                used = model.used()
                k = len(used)
                assert src == sorted(p for p in used if p >= k) and dst == [p for p in range(k) if p not in used]
                move = dict(zip(src, dst))
                model.seqs = {s: ([move.get(p, p) for p in pages], t) for s, (pages, t) in model.seqs.items()}
                assert model.used() == set(range(k))
            assert pool.free_pages == len(model.free())
            for s, (pages, t) in model.seqs.items():
                assert pool.pages(s) == pages and pool.length(s) == t
            table, lens = pool.block_table(model.seqs)
            for row, (pages, t) in zip(table.tolist(), model.seqs.values()):
                assert row[:len(pages)] == pages and set(row[len(pages):]) <= {-1}
            assert lens.tolist() == [t for _, t in model.seqs.values()]


def test_pool_refuses():
    h = ctypes.c_void_p()
    assert arf.arf_pages_create(-1, 4, h) == INVALID and arf.arf_pages_create(4, 0, h) == INVALID
    assert arf.arf_pages_destroy(None) == arf.ARF_OK
    out = ctypes.c_int32()
    for st in (arf.arf_pages_open(None, 1, out), arf.arf_pages_fork(None, 0, out), arf.arf_pages_close(None, 0),
               arf.arf_pages_free(None, out), arf.arf_pages_extend(None, 0, 1, out, out)):
        assert st == INVALID
    with arf.PagePool(4, 4) as pool:
        for call in (lambda: pool.open(-1), lambda: pool.extend(0, 1), lambda: pool.fork(0), lambda: pool.free(0),
                     lambda: pool.length(0)):
            with pytest.raises(arf.ArfError) as e:
                call()
            assert e.value.status == INVALID
        s = pool.open(5)
        for call in (lambda: pool.extend(s, -1), lambda: pool.extend(s, 2 ** 63 - 1), lambda: pool.fork(s + 1)):
            with pytest.raises(arf.ArfError) as e:
                call()
            assert e.value.status == INVALID
        with pytest.raises(ValueError):
            pool.block_table([s], width=1)
        t = pool.open(9 - 1)
        pool.free(s)  # pages 2, 3 in use
        n = ctypes.c_int32()
        one = (ctypes.c_int32 * 1)()
        assert arf.arf_pages_compact(pool.handle, one, one, 1, n) == INVALID and n.value == 2
        assert pool.pages(t) == [2, 3]
        src, dst = pool.compact()
        assert (src.tolist(), dst.tolist()) == ([2, 3], [0, 1]) and pool.pages(t) == [0, 1]
        assert [x.tolist() for x in pool.compact()] == [[], []]


def test_pool_from_several_threads():
    import threading
    with arf.PagePool(256, 4) as pool:
        def work(k):
            rng = random.Random(k)
            for _ in range(200):
                s = pool.open(rng.randint(0, 20))
                c = pool.fork(s)
                pool.extend(c, 1)
                pool.free(s)
                pool.free(c)
        ts = [threading.Thread(target=work, args=(k,)) for k in range(4)]
        [t.start() for t in ts]
        [t.join() for t in ts]
        assert pool.free_pages == 256
        assert np.array_equal(pool.pages(pool.open(12)), [0, 1, 2])


def test_handles_do_not_change_under_their_structs():
    """A table's struct holds an address: what it is made of is not replaced."""
    t = arf.RotaryTable(8, device="cpu")
    for name, value in (("turns", t.turns.clone()), ("rot_dim", 4), ("layout", "interleaved"), ("magnitude", 2.0),
                        ("struct", None)):
        with pytest.raises(AttributeError):
            setattr(t, name, value)
    assert t.struct.turns == t.turns.data_ptr() and t.struct.rot_dim == t.rot_dim
    for name in ("k", "v", "layout", "dtype", "device", "num_pages", "page_size", "kv_heads", "head_dim", "struct"):
        assert getattr(arf.KVCache, name).fset is None


@pytest.mark.parametrize("seed", range(40))
def test_shared_elements_are_found(seed):
    """_share against the sets of bytes, for page tensors of every layout and
    offsets around those at which they begin to touch."""
    from all_reduce_residual_gb300.attention import _share
    rng = random.Random(seed)
    sizes = [rng.randint(1, 4) for _ in range(3)]
    row, inside, dims = rng.randint(1, 5), 0, []
    inside = row
    for n in sizes:  # each step beyond everything inside it
        stride = inside + rng.choice([0, 0, 1, rng.randint(0, 9)])
        dims.append((stride, n))
        inside += stride * (n - 1)
    rng.shuffle(dims)
    at = {sum(i * s for i, (s, _) in zip(index, dims)) + d
          for index in np.ndindex(*[n for _, n in dims]) for d in range(row)}
    for delta in range(-inside - 3, inside + 4):
        assert _share(delta, dims, row) == bool(at & {x + delta for x in at}), (delta, dims, row)
    assert not _share(0, [(8, 0), (4, 2), (2, 2)], 2)


def test_numbers_are_not_cut_off():
    """Integers beyond the C types are refused, not taken modulo 2^32 or 2^64."""
    for make in (lambda: arf.PagePool((1 << 32) + 4, 4), lambda: arf.PagePool(4, (1 << 32) + 4),
                 lambda: arf.RotaryTable((1 << 32) + 8, device="cpu"), lambda: arf.RotaryTable((1 << 20) + 2, device="cpu"),
                 lambda: arf.KVCache(*[torch.zeros(1, 1, 1, 8, dtype=torch.bfloat16).expand((1 << 32) + 4, -1, -1, -1)] * 2)):
        with pytest.raises(ValueError):
            make()
    with arf.PagePool(8, 4) as pool:
        s = pool.open(3)
        big = s + (1 << 32)
        for call in (lambda: pool.open((1 << 64) + 1), lambda: pool.extend(s, (1 << 64) + 1), lambda: pool.extend(big, 1),
                     lambda: pool.fork(big), lambda: pool.free(big), lambda: pool.length(big), lambda: pool.pages(big),
                     lambda: pool.block_table([big])):
            with pytest.raises(ValueError):
                call()
        with pytest.raises(TypeError):
            pool.open(2.0)
        assert pool.length(s) == 3 and pool.free_pages == 7


def test_table_of_given_frequencies():
    for base, rot in ((10000.0, 64), (500000.0, 6)):
        w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
        a, b = arf.RotaryTable(rot, base=base, device="cpu"), arf.RotaryTable.from_frequencies(w, device="cpu")
        # the same binary64 frequencies, a division and a product by 2^64 each
        assert all(abs(x - y) <= abs(x) * 2.0 ** -50 + 1 for x, y in zip(a.turns.tolist(), b.turns.tolist()))
        assert (b.rot_dim, b.layout, b.magnitude) == (rot, "half", 1.0) and b.struct.rot_dim == rot
    t = arf.RotaryTable.from_frequencies(torch.tensor([-0.5, 0.0, 7.0], dtype=torch.float64), 0.75, "interleaved", "cpu")
    want = [x / (2 * math.pi) % 1.0 for x in (-0.5, 0.0, 7.0)]  # whole turns drop out
    got = [x % 2 ** 64 / 2.0 ** 64 for x in t.turns.tolist()]
    assert all(abs(x - y) <= 2.0 ** -52 for x, y in zip(got, want))
    assert t.struct.interleaved == 1 and t.struct.magnitude == 0.75 and t.rot_dim == 6
    for bad in (dict(frequencies=[]), dict(frequencies=[1.0, math.inf]), dict(frequencies=[math.nan]),
                dict(frequencies=[1.0], magnitude=math.inf), dict(frequencies=[1.0], layout="other")):
        with pytest.raises(ValueError):
            arf.RotaryTable.from_frequencies(**bad, device="cpu")
