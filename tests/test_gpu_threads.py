"""Calls of different sizes from several host threads at once: what one thread
asks of a kernel's shared memory does not take another's launch away."""
import ctypes
import subprocess
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"

# n calls in a row with nothing of Python between them -> how many gave a status other than 0
COMBINE = """
typedef int (*call)(const void *, const void *, const void *, const void *, int, int, int, long long, void *, void *,
                    void *, void *, void *);
int many(call f, int n, const void *dy, const void *gates, const void *out, const void *slots, int T, int k, int d,
         void *q, void *s, void *dg, void *stream)
{
    int wrong = 0;
    for (int i = 0; i < n; i++) wrong += f(dy, gates, out, slots, T, k, d, (long long)T * k, q, s, dg, 0, stream) != 0;
    return wrong;
}
"""

ROUTE = """
typedef int (*call)(const void *, const void *, int, int, int, int, int, int, float, void *, void *, void *, void *, void *);
int many(call f, int n, const void *x, const void *w, int T, int d, int E, int k, void *ids, void *gates, void *stream)
{
    int wrong = 0;
    for (int i = 0; i < n; i++) wrong += f(x, w, T, d, E, k, 0, 1, 1.0f, ids, gates, 0, 0, stream) != 0;
    return wrong;
}
"""


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def loop_of(source, folder):
    (folder / "many.c").write_text(source)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", str(folder / "many.so"), str(folder / "many.c")], check=True)
    return ctypes.CDLL(str(folder / "many.so")).many


def together(calls):
    """Every call on a thread and a stream of its own -> what they returned."""
    got = [None] * len(calls)
    start = threading.Barrier(len(calls))

    def work(i):
        stream = torch.cuda.Stream()
        start.wait()
        got[i] = calls[i](stream)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return got


def test_combine_backward_of_different_widths(L, tmp_path):
    many = loop_of(COMBINE, tmp_path)
    fn = ctypes.cast(L._lib.moe_combine_backward, ctypes.c_void_p)
    g = torch.Generator(device=DEV).manual_seed(0)
    T, k = 8, 2

    def of(d):
        dy, out = (torch.randn(n, d, device=DEV, generator=g).bfloat16() for n in (T, T * k))
        gates = torch.rand(T, k, device=DEV, generator=g)
        sl2 = torch.randperm(T * k, device=DEV, generator=g).int()
        bufs = [(torch.empty(T * k, d, dtype=torch.uint8, device=DEV), torch.empty(T * k, d // 128, device=DEV),
                 torch.empty(T, k, device=DEV)) for _ in range(2)]
        L.moe_combine_backward(dy, gates, out, sl2, *bufs[0])
        P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        call = lambda stream: many(fn, 3000, P(dy), P(gates), P(out), P(sl2), T, k, d, *map(P, bufs[1]),  # noqa: E731
                                   ctypes.c_void_p(stream.cuda_stream))
        return call, bufs, (dy, gates, out, sl2)

    made = [of(d) for d in (128, 8192, 4096, 7168)]
    assert together([m[0] for m in made]) == [0] * 4
    for _, (want, got), _ in made:
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_route_of_different_experts(L, tmp_path):
    many = loop_of(ROUTE, tmp_path)
    fn = ctypes.cast(L._lib.moe_route_topk, ctypes.c_void_p)
    g = torch.Generator(device=DEV).manual_seed(1)
    T, d = 64, 128

    def of(E, k):
        x, w = (torch.randn(n, d, device=DEV, generator=g).bfloat16() for n in (T, E))
        bufs = [(torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)) for _ in range(2)]
        L.moe_route_topk(x, w, k, 0, topk_ids=bufs[0][0], topk_gates=bufs[0][1])
        P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        call = lambda stream: many(fn, 3000, P(x), P(w), T, d, E, k, *map(P, bufs[1]),  # noqa: E731
                                   ctypes.c_void_p(stream.cuda_stream))
        return call, bufs, (x, w)

    made = [of(8, 2), of(1024, 32), of(256, 8), of(1024, 8)]
    assert together([m[0] for m in made]) == [0] * 4
    for _, (want, got), _ in made:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
