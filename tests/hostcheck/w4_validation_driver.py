"""Drives the C-ABI layer of the 4-bit products, the router and the experts built for the host with AddressSanitizer
and UndefinedBehaviorSanitizer (w4_api.hip and the stub launchers beside this file), without a GPU and without torch.
Argument: the sanitized library.  Known statuses, the choice of forms, then a seeded random sweep: every status is a
defined one, a call that returns an error has launched nothing, and no product is launched in a form that does not fit."""
import ctypes
import random
import sys

lib = ctypes.CDLL(sys.argv[1])
P, I64, I32, S, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float


class Weight(ctypes.Structure):
    _fields_ = [("q_w", P), ("s_w", P), ("z_w", P), ("n", I64)]


SIG = {
    "qlin_pack_w4": [P, P, P, I64, I64, I64, I32, P, P, P, P],
    "qlin_linear_w4": [P, I64, I64, I32, P, P, I32, S, P],
    "qlin_linear_swiglu_w4": [P, I64, I64, I32, P, P, P, P],
    "qlin_route": [P, S, I64, I64, I32, S, P, I32, I32, I32, I32, F, P, P, P],
    "qlin_experts_w4": [P, I64, I64, I64, I64, I32, I32, P, P, P, P, P, P, P, P],
}
for name, args in SIG.items():
    getattr(lib, name).restype = S
    getattr(lib, name).argtypes = args
lib.qlin_w4_packed_bytes.restype = lib.qlin_w4_packed_scales.restype = lib.qlin_experts_w4_workspace.restype = I64
lib.qlin_w4_packed_bytes.argtypes = [I64, I64]
lib.qlin_w4_packed_scales.argtypes = [I64, I64, I32]
lib.qlin_experts_w4_workspace.argtypes = [I64, I32, I64, I64, I64]
lib.w4_items.restype = ctypes.c_longlong

OK, NULL, SHAPE, ALIGN, UNSUP, HIP, ALIAS = range(7)
A = 0x10000000000          # fake addresses far apart: never dereferenced
GIB = 1 << 32
calls = 0


def at(i, off=0):
    return A + i * GIB + off


def call(name, *args):
    global calls
    before = lib.w4_launches()
    st = getattr(lib, name)(*args)
    assert st in (OK, NULL, SHAPE, ALIGN, UNSUP, ALIAS), (name, st)
    if st != OK:
        assert lib.w4_launches() == before, f"{name} returned {st} after launching"
    assert not lib.w4_bad(), (name, args)
    calls += 1
    return st


def weights(*items):
    """An array of exactly len(items) entries, in memory that ends there."""
    arr = (Weight * max(1, len(items)))()
    for i, w in enumerate(items):
        arr[i] = Weight(*w)
    return arr


def pointers(*items):
    return (P * max(1, len(items)))(*items)


def linear(M, K, group, ws, ys, nw=None, out=0, x=at(0)):
    return call("qlin_linear_w4", x, M, K, group, weights(*ws), pointers(*ys), len(ws) if nw is None else nw, out, None)


# ---- known statuses --------------------------------------------------------
w = (at(1), at(2), None, 256)
assert linear(4, 256, 128, [w], [at(4)]) == OK
assert linear(0, 256, 128, [w], [at(4)]) == OK
assert linear(4, 256, 128, [(None, None, None, 0)], [None]) == OK
assert linear(4, 256, 128, [w], [at(4)], nw=0) == SHAPE
assert linear(4, 256, 128, [w], [at(4)], nw=5) == SHAPE
assert linear(4, 250, 128, [w], [at(4)]) == SHAPE          # K % 32
assert linear(4, 288, 128, [w], [at(4)]) == SHAPE          # K % group
assert linear(4, 256, 16, [w], [at(4)]) == SHAPE
assert linear(4, 131104, 32, [w], [at(4)]) == SHAPE
assert linear(-1, 256, 128, [w], [at(4)]) == SHAPE
assert linear(4, 256, 128, [w], [at(4)], out=1) == UNSUP
assert linear(4, 256, 128, [w], [at(4)], x=None) == NULL
assert linear(4, 256, 128, [(None, at(2), None, 256)], [at(4)]) == NULL
assert linear(4, 256, 128, [w], [None]) == NULL
assert linear(4, 256, 128, [(at(1, 8), at(2), None, 256)], [at(4)]) == ALIGN
assert linear(4, 256, 128, [(at(1), at(2, 2), None, 256)], [at(4)]) == ALIGN
assert linear(4, 256, 128, [(at(1), at(2), at(3, 2), 256)], [at(4)]) == ALIGN
assert linear(4, 256, 128, [w], [at(4, 8)]) == ALIGN
assert linear(4, 256, 128, [w], [at(1, 64)]) == ALIAS      # y in the codes
assert linear(4, 256, 128, [w], [at(2, 64)]) == ALIAS      # y in the scales
assert linear(4, 256, 128, [(at(1), at(2), at(3), 256)], [at(3, 16)]) == ALIAS
assert linear(4, 256, 128, [w], [at(0, 1024)]) == ALIAS    # y in x
assert linear(4, 256, 128, [w, w], [at(4), at(4, 512)]) == ALIAS
assert linear(4, 256, 128, [w, w], [at(4), at(5)]) == OK   # one matrix twice
assert linear(1 << 24, 131072, 128, [(at(1), at(2), None, 1 << 24)], [at(4)]) == SHAPE

assert lib.qlin_w4_packed_bytes(17, 160) == 2 * 2 * 1024
assert lib.qlin_w4_packed_bytes(0, 128) == 0 and lib.qlin_w4_packed_bytes(16, 100) == 0
assert lib.qlin_w4_packed_scales(17, 160, 32) == 2 * 2 * 16 * 4


def pack(E=2, N=40, K=160, group=32, q=at(0), s=at(1), z=at(2), qp=at(3), sp=at(4), zp=at(5)):
    return call("qlin_pack_w4", q, s, z, E, N, K, group, qp, sp, zp, None)


assert pack() == OK and pack(z=None, zp=None) == OK and pack(N=0, q=None) == OK
assert pack(z=None) == NULL and pack(zp=None) == NULL and pack(q=None) == NULL
assert pack(E=1025) == SHAPE and pack(group=64) == SHAPE and pack(K=96 + 16) == SHAPE and pack(N=-1) == SHAPE
assert pack(q=at(0, 4)) == ALIGN and pack(sp=at(4, 4)) == ALIGN
assert pack(qp=at(0, 160)) == ALIAS and pack(sp=at(3, 1024)) == ALIAS


def swiglu(M=4, K=256, group=64, gate=(at(1), at(2), None, 48), up=(at(3), at(4), at(5), 48), h=at(6), x=at(0)):
    return call("qlin_linear_swiglu_w4", x, M, K, group, weights(gate) if gate else None, weights(up), h, None)


assert swiglu() == OK and swiglu(M=0) == OK
assert swiglu(gate=None) == NULL and swiglu(h=None) == NULL
assert swiglu(up=(at(3), at(4), None, 64)) == SHAPE and swiglu(K=224) == SHAPE
assert swiglu(h=at(6, 8)) == ALIGN and swiglu(h=at(5)) == ALIAS and swiglu(h=at(0, 16)) == ALIAS


def route(T=4, E=64, k=8, ltype=2, score=0, bias=at(1), groups=8, top=4, best=2, logits=at(0), ids=at(2), wt=at(3)):
    return call("qlin_route", logits, ltype, T, E, k, score, bias, groups, top, best, 1, 1.0, ids, wt, None)


assert route() == OK and route(T=0) == OK and route(bias=None) == OK and route(ltype=0) == OK
assert route(k=33) == SHAPE and route(k=0) == SHAPE and route(E=1025) == SHAPE and route(E=0) == SHAPE
assert route(groups=7) == SHAPE and route(groups=0) == SHAPE and route(top=9) == SHAPE and route(top=0) == SHAPE
assert route(E=64, groups=64, top=4) == SHAPE              # k past the experts of the groups that stay
assert route(E=128, groups=128) == SHAPE and route(best=3) == SHAPE
assert route(ltype=1) == UNSUP and route(score=2) == UNSUP
assert route(logits=None) == NULL and route(ids=None) == NULL and route(wt=None) == NULL
assert route(logits=at(0, 2)) == ALIGN and route(logits=at(0, 2), ltype=0) == OK and route(ids=at(2, 1)) == ALIGN
assert route(ids=at(0, 4)) == ALIAS and route(wt=at(2, 64)) == ALIAS and route(wt=at(1)) == ALIAS


def experts(T=8, H=256, I=128, E=16, k=4, group=64, x=at(0), ids=at(1), wt=at(2), y=at(12), work=at(13), gate=None, up=None,
            down=None):
    gate = (at(3), at(4), None, I) if gate is None else gate
    up = (at(5), at(6), None, I) if up is None else up
    down = (at(7), at(8), at(9), H) if down is None else down
    return call("qlin_experts_w4", x, T, H, I, E, k, group, ids, wt, weights(gate), weights(up), weights(down), y, work, None)


assert experts() == OK and experts(T=0) == OK and experts(T=500) == OK
assert experts(k=33) == SHAPE and experts(k=0) == SHAPE and experts(E=0) == SHAPE and experts(E=1025) == SHAPE
assert experts(H=250) == SHAPE and experts(I=96) == SHAPE and experts(T=1 << 24) == SHAPE
assert experts(gate=(at(3), at(4), None, 64)) == SHAPE and experts(down=(at(7), at(8), None, 128)) == SHAPE
assert experts(x=None) == NULL and experts(work=None) == NULL and experts(up=(at(5), None, None, 128)) == NULL
assert experts(y=at(12, 8)) == ALIGN and experts(work=at(13, 8)) == ALIGN and experts(ids=at(1, 2)) == ALIGN
assert experts(y=at(0, 64)) == ALIAS and experts(work=at(7)) == ALIAS and experts(y=at(13)) == ALIAS
assert experts(work=at(2, -64)) == ALIAS
assert lib.qlin_experts_w4_workspace(8, 4, 16, 250, 128) == 0 and lib.qlin_experts_w4_workspace(0, 4, 16, 256, 128) == 0
assert lib.qlin_experts_w4_workspace(8, 4, 16, 256, 128) >= 8 * 4 * 128 * 4

sizes = [lib.qlin_experts_w4_workspace(T, 2, 16, 1024, 512) for T in range(1, 200)]
assert sizes == sorted(sizes)                            # a workspace serves any fewer tokens

# ---- the choice of forms: 16 x 1, 16 x 2, 16 x 4 (eight or four wavefronts), 32 x 4, tiled 64 x 8, 64 x 16 ----
big = lambda n: (at(1), at(2), None, n)  # noqa: E731
for M, N, K, form in [(1, 4096, 4096, 0), (1, 14336, 4096, 3), (32, 4096, 4096, 1), (64, 4096, 4096, 3), (128, 4096, 4096, 4),
                      (512, 4096, 4096, 5), (2048, 4096, 4096, 6), (2048, 4096, 14336, 6), (333, 1488, 2048, 3)]:
    assert linear(M, K, 128, [big(N)], [at(4)]) == OK
    assert lib.w4_form() == form, (M, N, K, lib.w4_form())

# ---- seeded random sweep ---------------------------------------------------
rng = random.Random(20261206)
SIZES = [0, 1, 2, 5, 16, 17, 33, 64, 65, 500, 4096, 14336, 131072, 1 << 20, 1 << 24, (1 << 24) + 1, -1, 1 << 40]


def ptr():
    r = rng.random()
    if r < 0.03:
        return None
    if r < 0.08:
        return at(rng.randrange(40), rng.choice([1, 2, 4, 8]))
    if r < 0.13:
        return at(0, rng.randrange(1 << 20) * 16)
    return at(rng.randrange(40))


def size():
    return rng.choice(SIZES) if rng.random() < 0.5 else rng.randrange(1, 5000)


def weight(n):
    return (ptr(), ptr(), ptr() if rng.random() < 0.4 else None, n)


for it in range(20000):
    K, group = rng.choice([32, 128, 160, 1024, 4096, 14336, 131072, 100, 0, -32, 131104]), rng.choice([32, 64, 128, 128, 16, 0])
    fn = rng.randrange(5)
    if fn == 0:
        n = rng.randrange(0, 6)
        cnt = n if rng.random() < 0.8 else rng.choice([0, 5, -1])
        linear(size(), K, group, [weight(size()) for _ in range(n)], [ptr() for _ in range(n)],
               nw=cnt if n or cnt <= 0 or cnt > 4 else 0, out=rng.choice([0, 0, 2, 1, 7]), x=ptr())
    elif fn == 1:
        n = size()
        swiglu(size(), K, group, weight(n), weight(n if rng.random() < 0.8 else size()), ptr(), ptr())
    elif fn == 2:
        route(size(), rng.choice([1, 8, 60, 256, 1024, 1025, 0]), rng.randrange(-1, 34), rng.choice([0, 2, 1]), rng.randrange(0, 3),
              ptr(), rng.choice([1, 1, 2, 4, 8, 64, 65, 0]), rng.randrange(0, 9), rng.randrange(0, 4), ptr(), ptr(), ptr())
    elif fn == 3:
        pack(rng.choice([0, 1, 4, 1024, 1025]), size(), K, group, *[ptr() for _ in range(6)])
    else:
        I = rng.choice([32, 128, 736, 1024, 4096, 100])
        experts(size(), K, I, rng.choice([1, 8, 64, 1024, 0]), rng.randrange(0, 34), group, ptr(), ptr(), ptr(), ptr(), ptr(),
                weight(I), weight(I), weight(K))

print(f"w4 hostcheck: {calls} calls, {lib.w4_launches()} launches, no sanitizer report")
