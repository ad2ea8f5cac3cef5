"""Drives the C-ABI layer of the norm, rotary, cache and attention calls built for the host with AddressSanitizer and
UndefinedBehaviorSanitizer (layer_api.hip and the stub launchers beside this file), without a GPU and without torch.
Argument: the sanitized library.  Known statuses, then a seeded random sweep: every status is a defined one, a call that
returns an error has launched nothing, and nothing is launched that a kernel does not take."""
import ctypes
import math
import random
import sys

lib = ctypes.CDLL(sys.argv[1])
P, I64, I32, S, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float


class Rotation(ctypes.Structure):
    _fields_ = [("frequencies", P), ("dims", I32), ("interleaved", I32), ("strength", F)]


class Cache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("pages", I64), ("kv_heads", I32), ("page_size", I32), ("dim", I32),
                ("kind", I32)]


class Queries(ctypes.Structure):
    _fields_ = [("q", P), ("stride", I64), ("gamma", P), ("out", P), ("out_stride", I64), ("heads", I32)]


SIG = {
    "qlin_norm_bf16": [P, P, P, I64, I64, F, P, P, P],
    "qlin_norm_int8": [P, P, P, I64, I64, F, P, P, P, P],
    "qlin_norm_fp8": [P, P, P, I64, I64, F, I32, P, P, P, P],
    "qlin_rope": [P, I64, P, I64, I32, I32, P, P, F, P, I64, P],
    "qlin_cache_write": [P, P, I64, P, I64, P, I64, P, P, P, F, P, P],
    "qlin_cache_read": [P, P, I64, P, P, P],
    "qlin_attn_decode": [P, P, P, I64, I32, I64, P, I64, F, P, P, P],
}
for name, args in SIG.items():
    getattr(lib, name).restype = S
    getattr(lib, name).argtypes = args
lib.qlin_attn_decode_workspace.restype = I64
lib.qlin_attn_decode_workspace.argtypes = [I32, I32, I32]

OK, NULL, SHAPE, ALIGN, UNSUP, HIP, ALIAS = range(7)
A = 0x10000000000          # fake addresses far apart: never dereferenced
FAR = 1 << 56
calls = 0


def at(i, off=0):
    return A + (i << 50) + off


def call(name, *args):
    global calls
    before = lib.layer_launches()
    st = getattr(lib, name)(*[ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args])
    assert st in (OK, NULL, SHAPE, ALIGN, UNSUP, ALIAS), (name, st)
    if st != OK:
        assert lib.layer_launches() == before, f"{name} returned {st} after launching"
    assert not lib.layer_bad(), (name, args)
    calls += 1
    return st


def expect(want, name, *args):
    got = call(name, *args)
    assert got == want, (name, args, got, want)


def cache(k=at(20), v=at(21), ks=at(22), vs=at(23), pages=7, kv=4, page=32, dim=64, kind=1):
    return Cache(k, v, ks, vs, pages, kv, page, dim, kind)


# ---- norm -----------------------------------------------------------------
x, r, g, t, y, s = (at(i) for i in range(6))
expect(OK, "qlin_norm_int8", x, r, g, 4, 64, 1e-6, t, y, s, None)
expect(OK, "qlin_norm_int8", x, None, g, 4, 64, 1e-6, None, y, s, None)
expect(OK, "qlin_norm_int8", x, r, g, 4, 64, 1e-6, r, y, s, None)            # in place
expect(OK, "qlin_norm_int8", x, r, g, 4, 64, 1e-6, x, y, s, None)
expect(OK, "qlin_norm_int8", None, None, None, 0, 64, 1e-6, None, None, None, None)
expect(NULL, "qlin_norm_int8", x, r, g, 4, 64, 1e-6, None, y, s, None)
expect(NULL, "qlin_norm_int8", x, None, g, 4, 64, 1e-6, t, y, s, None)
expect(NULL, "qlin_norm_int8", x, None, g, 4, 64, 1e-6, None, y, None, None)
expect(NULL, "qlin_norm_int8", x, None, None, 4, 64, 1e-6, None, y, s, None)
expect(SHAPE, "qlin_norm_int8", x, None, g, 4, 72, 1e-6, None, y, s, None)
expect(SHAPE, "qlin_norm_int8", x, None, g, 4, 131072 + 16, 1e-6, None, y, s, None)
expect(SHAPE, "qlin_norm_int8", x, None, g, -1, 64, 1e-6, None, y, s, None)
expect(UNSUP, "qlin_norm_int8", x, None, g, 4, 64, 0.0, None, y, s, None)
expect(UNSUP, "qlin_norm_int8", x, None, g, 4, 64, math.nan, None, y, s, None)
expect(ALIGN, "qlin_norm_int8", x + 8, None, g, 4, 64, 1e-6, None, y, s, None)
expect(ALIGN, "qlin_norm_int8", x, None, g, 4, 64, 1e-6, None, y, s + 2, None)
expect(ALIAS, "qlin_norm_int8", x, r, g, 4, 64, 1e-6, r + 128, y, s, None)     # half over the residual
expect(ALIAS, "qlin_norm_int8", x, None, g, 4, 64, 1e-6, None, x + 256, s, None)
expect(ALIAS, "qlin_norm_int8", x, None, g, 4, 64, 1e-6, None, y, y + 252, None)
expect(ALIAS, "qlin_norm_bf16", x, r, g, 4, 64, 1e-6, t, t, None)
expect(ALIAS, "qlin_norm_bf16", x, r, g, 4, 64, 1e-6, g, y, None)
expect(SHAPE, "qlin_norm_fp8", x, None, g, 4, 64, 1e-6, 128, None, y, s, None)
expect(SHAPE, "qlin_norm_fp8", x, None, g, 4, 128, 1e-6, 64, None, y, s, None)
expect(OK, "qlin_norm_fp8", x, None, g, 4, 128, 1e-6, 128, None, y, s, None)

# ---- rotary ---------------------------------------------------------------
rot = Rotation(at(7), 32, 0, 1.0)
pos = at(8)
expect(OK, "qlin_rope", x, 256, pos, 5, 4, 64, rot, None, 0.0, y, 256, None)
expect(OK, "qlin_rope", x, 256, pos, 5, 4, 64, rot, None, 0.0, x, 256, None)
expect(OK, "qlin_rope", None, 256, None, 0, 4, 64, rot, None, 0.0, None, 256, None)
expect(ALIAS, "qlin_rope", x, 512, pos, 5, 4, 64, rot, None, 0.0, x, 256, None)
expect(OK, "qlin_rope", x, 512, pos, 5, 4, 64, rot, None, 0.0, x + 512, 512, None)     # the other half of the rows
expect(ALIAS, "qlin_rope", x, 512, pos, 5, 4, 64, rot, None, 0.0, x + 496, 512, None)
expect(ALIAS, "qlin_rope", x + 512, 512, pos, 5, 4, 64, rot, None, 0.0, x + 16, 512, None)
expect(OK, "qlin_rope", x + 512, 512, pos, 5, 4, 64, rot, None, 0.0, x, 512, None)
expect(SHAPE, "qlin_rope", x, 248, pos, 5, 4, 64, rot, None, 0.0, y, 256, None)
expect(SHAPE, "qlin_rope", x, 260, pos, 5, 4, 64, rot, None, 0.0, y, 256, None)
expect(SHAPE, "qlin_rope", x, 256, pos, 5, 4, 72, rot, None, 0.0, y, 256, None)
expect(SHAPE, "qlin_rope", x, 2048, pos, 5, 4, 272, rot, None, 0.0, y, 2048, None)
expect(SHAPE, "qlin_rope", x, 256, pos, 5, 0, 64, rot, None, 0.0, y, 256, None)
expect(SHAPE, "qlin_rope", x, 256, pos, 5, 4, 64, Rotation(at(7), 80, 0, 1.0), None, 0.0, y, 256, None)
expect(SHAPE, "qlin_rope", x, 256, pos, 5, 4, 64, Rotation(at(7), 24, 0, 1.0), None, 0.0, y, 256, None)
expect(NULL, "qlin_rope", x, 256, pos, 5, 4, 64, None, None, 0.0, y, 256, None)
expect(NULL, "qlin_rope", x, 256, None, 5, 4, 64, rot, None, 0.0, y, 256, None)
expect(NULL, "qlin_rope", x, 256, pos, 5, 4, 64, Rotation(None, 32, 0, 1.0), None, 0.0, y, 256, None)
expect(ALIGN, "qlin_rope", x, 256, pos, 5, 4, 64, Rotation(at(7) + 4, 32, 0, 1.0), None, 0.0, y, 256, None)
expect(UNSUP, "qlin_rope", x, 256, pos, 5, 4, 64, Rotation(at(7), 32, 2, 1.0), None, 0.0, y, 256, None)
expect(UNSUP, "qlin_rope", x, 256, pos, 5, 4, 64, Rotation(at(7), 32, 0, math.inf), None, 0.0, y, 256, None)
expect(UNSUP, "qlin_rope", x, 256, pos, 5, 4, 64, rot, g, 0.0, y, 256, None)
expect(ALIAS, "qlin_rope", x, 256, y + 64, 5, 4, 64, rot, None, 0.0, y, 256, None)

# ---- cache ----------------------------------------------------------------
slots, k, v, q, o = at(9), at(10), at(11), at(12), at(13)


def w(want, c=None, T=5, slots=slots, k=k, ks=256, v=v, vs=256, pos=pos, rot=rot, kg=None, eps=0.0, qs=None):
    expect(want, "qlin_cache_write", c or cache(), slots, T, k, ks, v, vs, pos, rot, kg, eps, qs, None)


w(OK)
w(OK, rot=None, pos=None)
w(OK, qs=Queries(q, 512, None, o, 512, 8))
w(OK, qs=Queries(q, 512, None, q, 512, 8))
w(OK, k=q + 1024, ks=1024, v=q + 1536, vs=1024, qs=Queries(q, 1024, None, q, 1024, 8))     # one projection's rows, in place
w(ALIAS, k=q + 1008, ks=1024, v=q + 1536, vs=1024, qs=Queries(q, 1024, None, q, 1024, 8))
w(ALIAS, qs=Queries(q, 512, None, k, 512, 8))
w(NULL, rot=None, pos=None, qs=Queries(q, 512, None, o, 512, 8))
w(OK, rot=None, pos=None, eps=1e-5, qs=Queries(q, 512, g, o, 512, 8))
w(UNSUP, rot=None, pos=None, eps=2.0, qs=Queries(q, 512, g, o, 512, 8))
w(UNSUP, kg=g)
w(NULL, qs=Queries(None, 512, None, o, 512, 8))
w(NULL, pos=None)
w(NULL, slots=None)
w(NULL, k=None)
w(OK, T=0, slots=None, k=None, v=None)
w(SHAPE, T=-1)
w(SHAPE, ks=248)
w(SHAPE, qs=Queries(q, 504, None, o, 512, 8))
w(SHAPE, qs=Queries(q, 512, None, o, 512, 0))
w(SHAPE, cache(page=24))
w(SHAPE, cache(page=0))
w(SHAPE, cache(pages=0))
w(SHAPE, cache(pages=1 << 27))
w(SHAPE, cache(kv=0))
w(SHAPE, cache(dim=40))
w(UNSUP, cache(kind=3))
w(NULL, cache(ks=None))
w(OK, cache(kind=0, ks=None, vs=None))
w(NULL, cache(k=None))
w(ALIGN, cache(v=at(21, 8)))
w(ALIGN, cache(ks=at(22, 4)))
w(ALIAS, cache(v=at(20, 64)))
w(ALIAS, cache(ks=at(20, 16)))
w(ALIAS, cache(k=k + 256))
w(ALIAS, slots=at(20, 64))
expect(NULL, "qlin_cache_write", None, slots, 5, k, 256, v, 256, pos, rot, None, 0.0, None, None)
expect(OK, "qlin_cache_read", cache(), slots, 5, k, v, None)
expect(OK, "qlin_cache_read", cache(), None, 0, None, None, None)
expect(NULL, "qlin_cache_read", cache(), slots, 5, k, None, None)
expect(ALIAS, "qlin_cache_read", cache(), slots, 5, k, k + 128, None)
expect(ALIAS, "qlin_cache_read", cache(), slots, 5, at(22, 16), v, None)
expect(ALIGN, "qlin_cache_read", cache(), slots, 5, k + 2, v, None)
expect(SHAPE, "qlin_cache_read", cache(), slots, 1 << 25, k, v, None)

# ---- attention ------------------------------------------------------------
table, lengths, ws = at(14), at(15), at(16)


def a(want, c=None, q=q, table=table, S=3, heads=8, columns=10, lengths=lengths, window=0, scale=0.1, out=o, ws=ws):
    expect(want, "qlin_attn_decode", q, c or cache(), table, S, heads, columns, lengths, window, scale, out, ws, None)


a(OK)
a(OK, S=0, q=None, table=None, lengths=None, out=None, ws=None)
a(OK, columns=0, table=None)
a(NULL, table=None)
a(NULL, ws=None)
a(NULL, lengths=None)
a(SHAPE, heads=6)
a(SHAPE, heads=2)
a(SHAPE, window=-1)
a(OK, window=1 << 40)
a(SHAPE, columns=-1)
a(OK, columns=1 << 25)
a(SHAPE, columns=(1 << 25) + 1)
a(SHAPE, S=1 << 25)
a(UNSUP, scale=math.inf)
a(UNSUP, scale=math.nan)
a(ALIGN, out=o + 2)
a(ALIGN, ws=ws + 8)
a(ALIAS, out=q)
a(ALIAS, ws=o + 16)
a(ALIAS, out=at(20, 16))
expect(NULL, "qlin_attn_decode", q, None, table, 3, 8, 10, lengths, 0, 0.1, o, ws, None)
for bad in ((0, 1, 64), (8, 0, 64), (8, 3, 64), (8, 4, 24), (8, 4, 512), (2048, 1, 64)):
    assert lib.qlin_attn_decode_workspace(*bad) == 0, bad
assert lib.qlin_attn_decode_workspace(32, 8, 128) > 0

# ---- random sweep ---------------------------------------------------------
rng = random.Random(11)
MN = (1 << 24)


def size(*usual):
    return rng.choice(usual) if rng.random() < 0.85 else rng.choice((0, 1, -1, 16, MN, MN + 1, 1 << 31, -(1 << 31)))


def i32(*usual):
    return max(-(1 << 31), min((1 << 31) - 1, size(*usual)))


def ptr():
    return None if rng.random() < 0.05 else at(rng.randrange(200), rng.choice([0] * 40 + [8, 16, 256, 4096]))


def any_rotation():
    return rng.choice([None, Rotation(ptr(), i32(32, 64, 128), i32(0, 1), rng.choice([1.0, 1.2, math.nan]))])


def any_cache():
    return rng.choice([None] + 6 * [cache(ptr(), ptr(), ptr(), ptr(), size(5, 100), i32(2, 8), i32(16, 48), i32(64, 128), i32(0, 1, 2))])


launched = lib.layer_launches()
for _ in range(30000):
    eps = rng.choice([1e-6, 1e-5, 0.0, math.nan, 2.0])
    kind = rng.randrange(6)
    if kind == 0:
        call("qlin_norm_fp8", ptr(), ptr(), ptr(), size(3, 70), size(128, 4096, 48), eps, i32(0, 128), ptr(), ptr(), ptr(), None)
    elif kind == 1:
        call("qlin_norm_bf16", ptr(), ptr(), ptr(), size(3, 70), size(128, 4096, 48), eps, ptr(), ptr(), None)
    elif kind == 2:
        call("qlin_rope", ptr(), size(512, 1024), ptr(), size(3, 9), i32(4, 8), i32(64, 128), any_rotation(), ptr(), eps, ptr(), size(512, 1024),
             None)
    elif kind == 3:
        qs = rng.choice([None, Queries(ptr(), size(1024, 2048), ptr(), ptr(), size(1024, 2048), i32(8, 4))])
        call("qlin_cache_write", any_cache(), ptr(), size(3, 9), ptr(), size(1024, 2048), ptr(), size(1024, 2048), ptr(), any_rotation(), ptr(),
             eps, qs, None)
    elif kind == 4:
        call("qlin_cache_read", any_cache(), ptr(), size(3, 9), ptr(), ptr(), None)
    else:
        call("qlin_attn_decode", ptr(), any_cache(), ptr(), size(3, 9), i32(8, 32), size(7, 100), ptr(), size(0, 64), rng.choice([0.1, math.inf]),
             ptr(), ptr(), None)
        lib.qlin_attn_decode_workspace(i32(8, 32), i32(2, 8), i32(64, 128))
assert lib.layer_launches() > launched + 200, "the sweep reached too few launches"
print(f"{calls} calls, no sanitizer report")
