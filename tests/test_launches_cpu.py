"""What the expert and integer calls launch, seen on the host: the library is
loaded over a stub of the HIP runtime (hip_stub.cpp) in a process of its own, so
no device is touched and no pointer is read."""

import os
import subprocess
import sys

import pytest

from nf4_bit_weight_amd import _lib as L

HERE = os.path.dirname(os.path.abspath(__file__))
F32, BF16, I8 = 0, 1, 2
A = 0x10000

# (T, E, k, groups, top_groups): every width; those of 512 and more with several waves want more than 64 KB of LDS
ROUTE = [(20000, 8, 2, 1, 1), (20000, 64, 8, 8, 4), (20000, 200, 4, 4, 2), (20000, 512, 8, 8, 2), (20000, 1000, 3, 1, 1), (20000, 1024, 8, 1, 1),
         (4, 1024, 8, 1, 1), (2000, 900, 8, 3, 2)]
# (M, N, K): the forms for few rows, then every tile
PLAIN = [(1, 4096, 4096), (2, 4096, 4096), (16, 4096, 4096), (16, 8192, 4096), (16, 14336, 4096), (32, 4096, 4096), (32, 1024, 4096), (64, 8000, 1024),
         (200, 4096, 256), (512, 4096, 128), (1024, 4096, 640), (2048, 4096, 128), (4096, 4096, 256)]
GROUPED = [(40, 96, 384, 4), (3000, 1000, 256, 4), (6000, 2000, 256, 4)]

CHILD = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[3])
ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)                   # found before the runtime that the library names
lib = ctypes.CDLL(sys.argv[2])
import importlib.util
spec = importlib.util.spec_from_file_location("nf4_lib", sys.argv[4])
L = importlib.util.module_from_spec(spec)
sys.modules["nf4_lib"] = L
spec.loader.exec_module(L)
for name, (res, args) in L.SIGNATURES.items():
    getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
A, BIG = 0x10000, 1 << 40
flush = ctypes.CDLL(None).fflush
def say(text):
    flush(None)
    print(text, flush=True)
def route(T, E, k, g, tg, dt, bias=None, gs=0, plan=A):
    return lib.nf4_route_fwd(A, dt, E, T, E, k, bias, 1, g, tg, gs, 1, 1.0, A, A, plan, plan, plan, A, BIG, None)
def route_bwd(T, E, k, dt):
    return lib.nf4_route_bwd(A, A, dt, E, T, E, k, A, A, 0, 0, 1.0, A, None)
def plan(T, E, k):
    return lib.nf4_expert_plan(A, T, k, E, A, A, A, A, BIG, None)
def matmul(M, N, K, dt, out):
    return lib.nf4_int8_matmul(A, dt, K, A, M, A, A, N, K, None, A, out, A, BIG, None)
def grouped(M, N, K, E, dt, out):
    return lib.nf4_int8_grouped_matmul(A, dt, K, A, M, None, A, E, M, A, A, N, K, A, out, 1, A, BIG, None)
def rows(f, T, H, k, dt):
    a = {"gather": (A, dt, H, T, H, k, A, A, A, 1), "gather_bwd": (A, dt, T, H, k, A, A), "combine_fwd": (A, dt, T, H, k, A, A, A),
         "combine_bwd": (A, H, A, dt, T, H, k, A, A, A, A, A, 1)}[f]
    return getattr(lib, "nf4_expert_" + f)(*a, None)
def quantize(M, K, dt):
    return lib.nf4_int8_quantize(A, dt, K, M, K, A, A, None)
for line in sys.stdin:
    say("call " + line.strip())
    say("status %d" % eval(line))
"""


@pytest.fixture(scope="module")
def watch(tmp_path_factory):
    if not os.path.exists(L.LIB_PATH):
        from nf4_bit_weight_amd import build as B
        B.build()
    stub = str(tmp_path_factory.mktemp("stub") / "hip_stub.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", os.path.join(HERE, "hip_stub.cpp"), "-o", stub], check=True)

    def run(calls):
        """[(call, status, [(kernel, LDS, workgroups, threads each)])] and the limits raised, in order."""
        r = subprocess.run([sys.executable, "-c", CHILD, stub, L.LIB_PATH, HERE, L.__file__], input="\n".join(calls), capture_output=True,
                           text=True, timeout=100)
        assert r.returncode == 0, r.stderr[-2000:]
        names, limits, seen = {}, {}, []
        for line in r.stdout.splitlines():
            word, _, rest = line.partition(" ")
            if word == "kernel":
                names[rest.split()[0]] = rest.split()[1]
            elif word == "call":
                seen.append([rest, None, []])
            elif word == "status":
                seen[-1][1] = int(rest)
            elif word == "limit":
                f, n = rest.split()
                limits[f] = max(limits.get(f, 0), int(n))
            elif word == "launch":
                f, lds, x, y, z, threads = rest.split()
                seen[-1][2].append((names[f], int(lds), limits.get(f, 65536), int(x) * int(y) * int(z), int(threads)))
        assert len(seen) == len(calls)
        return seen
    return run


def every_call():
    calls = []
    for c in ROUTE:
        for dt in (F32, BF16):
            calls += [f"route({', '.join(map(str, c))}, {dt})", f"route({', '.join(map(str, c))}, {dt}, A)",
                      f"route({', '.join(map(str, c))}, {dt}, None, 1)", f"route_bwd({c[0]}, {c[1]}, {c[2]}, {dt})"]
        calls.append(f"plan({c[0]}, {c[1]}, {c[2]})")
    for c in PLAIN:
        calls += [f"matmul({', '.join(map(str, c))}, {dt}, {out})" for dt in (BF16, F32, I8) for out in (BF16, F32)]
    for c in GROUPED:
        calls += [f"grouped({', '.join(map(str, c))}, {dt}, {out})" for dt in (BF16, I8) for out in (BF16, F32)]
    return calls


@pytest.mark.parametrize("backwards", [False, True])
def test_every_kernel_may_have_its_lds(watch, backwards):
    """A kernel's limit on dynamic LDS (64 KB unless raised) is its own, whichever of its kind ran first."""
    calls = every_call()
    kernels = {}
    for call, status, launches in watch(calls[::-1] if backwards else calls):
        assert status == 0 and launches, call
        for name, lds, limit, groups, threads in launches:
            assert lds <= limit, f"{call}: {name} is launched with {lds} bytes, its limit is {limit}"
            assert lds <= 160 * 1024 and 0 < groups * threads < 2 ** 32 and threads <= 1024
            kernels[name] = max(lds, kernels.get(name, 0))
    for kind, many in (("k_route", 16), ("k_tile", 12), ("k_stream", 12)):
        assert sum(kind in n and not "bwd" in n for n in kernels) >= many, (kind, sorted(kernels))
    assert sum(lds > 65536 for lds in kernels.values()) >= 16


def sizes_at_the_limits():
    calls = []
    for E in (1, 8, 64, 100, 256, 257, 512, 513, 1024):
        for k in (1, 8, 64):
            for T in sorted({(1 << 30) // k, (1 << 26) - 1, (1 << 26) - 15, (1 << 26) - 16, 1 << 25, 1 << 24, (1 << 24) - 1} if k <= 16 else {(1 << 30) // k}):
                calls.append(f"plan({T}, {E}, {k})")
                if k > E:
                    continue
                calls += [f"route({T}, {E}, {k}, 1, 1, {BF16})", f"route({T}, {E}, {k}, 1, 1, {F32}, A)", f"route_bwd({T}, {E}, {k}, {F32})"]
                calls += [f"route({T}, {E}, {k}, {g}, 1, {F32}, A, 1)" for g in (2, 3) if E % g == 0]
    for T, H in ((1, 1 << 23), ((1 << 24) - 1, 256), ((1 << 24) - 1, 0), ((1 << 23) - 1, 512), (511, 1 << 23), (65536, 65535)):
        calls += [f"rows('{f}', {T}, {H}, {k}, {dt})" for f in ("gather", "gather_bwd", "combine_fwd", "combine_bwd") for k in (1, 64) for dt in (F32, BF16)]
    for M in (1, 16, 17, 64, 65, 1 << 20, (1 << 24) - 1, 1 << 28):
        calls.append(f"quantize({M}, 5000, {BF16})")
        for N in (64, 8191, 8192, 1 << 20, 59652288, 1 << 28):
            for K in (100, 300, 4096):
                calls += [f"matmul({M}, {N}, {K}, {dt}, 0)" for dt in (BF16, I8)] + [f"grouped({M}, {N}, {K}, {E}, 1, 1)" for E in (1, 1024)]
    return calls


def test_what_a_call_accepts_can_be_launched(watch):
    """Fewer than 2^32 threads in every launch, or the call is refused before the first of them."""
    accepted = 0
    for call, status, launches in watch(sizes_at_the_limits()):
        assert status == 0 if launches else status in (L.NF4_OK, L.NF4_ERR_UNSUPPORTED, L.NF4_ERR_WORKSPACE), call
        accepted += status == 0
        for name, lds, limit, groups, threads in launches:
            assert 0 < groups < 2 ** 31 and groups * threads < 2 ** 32 and lds <= limit, f"{call}: {name} {groups} x {threads}"
    assert accepted > 300


def test_sizes_that_fit_are_taken(watch):
    """The refusals stay close to what a launch holds."""
    calls = [f"route({(1 << 26) - 1}, 256, 8, 1, 1, {BF16})", f"route({(1 << 26) - 16}, 1024, 1, 1, 1, {BF16})",
             f"route({(1 << 26) - 16}, 513, 1, 3, 1, {BF16})", f"route_bwd({(1 << 26) - 16}, 1024, 1, {BF16})", f"plan({(1 << 26) - 16}, 1024, 1)"]
    assert [status for _, status, _ in watch(calls)] == [0] * len(calls)
    refused = [f"route({(1 << 26) - 15}, 257, 1, 1, 1, {BF16})", f"route_bwd({(1 << 26) - 1}, 1024, 1, {BF16})", f"plan({(1 << 26) - 1}, 1024, 1)",
               f"route({1 << 26}, 64, 1, 1, 1, {BF16})"]
    assert [(status, launches) for _, status, launches in watch(refused)] == [(L.NF4_ERR_UNSUPPORTED, [])] * len(refused)
