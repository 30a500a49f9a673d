"""Calls of the 8-bit KV cache that follow one another on a stream without the
host between them: every kernel may be set up while the one before it still
writes what it reads. The results are those of the same calls with a
synchronisation after each, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
B, HQ, HKV, D, L, BLOCK, STEPS = 5, 8, 4, 128, 900, 16, 10


def _serve(m, fmt, news, mode):
    """STEPS steps from inside open blocks, each with larger values than the last
    (so scales grow): tokens and queries arrive by copies on the stream, the
    tables advance on the device. Returns every step's outputs and the bytes of
    the positions held in the end."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    T = sum(news)
    i32 = dict(dtype=torch.int32, device=DEV)
    dims = dict(Hq=HQ, Hkv=HKV, D=D, L_max=L, block=BLOCK, format=fmt)
    sh = m.kv8_shape(B, T, **dims)
    held = [7, 1, 0, 13, 21]
    first = m.kv8_shape(B, sum(held), **dims)
    cache = m.kv8_alloc_cache(sh, DEV)
    off = torch.tensor([sum(news[:i]) for i in range(B + 1)], **i32)
    off0 = torch.tensor([sum(held[:i]) for i in range(B + 1)], **i32)
    add = torch.tensor(news, **i32)
    starts0 = torch.tensor(held, **i32)

    def values(n, heads, size=1.0):
        return (torch.randn(n, heads, D, generator=gen, device=DEV) * size).to(torch.bfloat16)

    k0, v0 = values(sum(held), HKV, 0.1), values(sum(held), HKV, 0.1)
    ks, vs = ([values(T, HKV, 1.3 ** i) for i in range(STEPS)] for _ in range(2))
    qs = [values(T, HQ, 1.3 ** -i) for i in range(STEPS)]
    k, v, q = torch.zeros_like(ks[0]), torch.zeros_like(vs[0]), torch.zeros_like(qs[0])
    starts, lens = torch.zeros_like(starts0), torch.zeros_like(starts0)
    ws = m.kv8_alloc_workspace(sh, DEV)
    o, ko, vo = (torch.empty(STEPS, *s.shape, dtype=torch.bfloat16, device=DEV) for s in (q, k, v))
    begin = torch.zeros(B, **i32)
    pause = torch.cuda.synchronize if mode == "sync" else lambda: None

    def steps():
        starts.copy_(starts0)
        torch.add(starts0, add, out=lens)
        m.kv8_write(first, k0, v0, off0, begin, cache)
        pause()
        for i in range(STEPS):
            k.copy_(ks[i]), v.copy_(vs[i]), q.copy_(qs[i])
            pause()
            m.kv8_write(sh, k, v, off, starts, cache)
            pause()
            m.kv8_read(sh, cache, off, starts, ko[i], vo[i])
            pause()
            m.kv8_attn(sh, q, cache, off, lens, o[i], ws)
            pause()
            starts.add_(add), lens.add_(add)
            pause()

    if mode == "graph":
        steps()  # the first calls set attributes
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            steps()
        for t in (o, ko, vo):
            t.zero_()
        g.replay()
    else:
        torch.cuda.synchronize()
        if mode == "queue":
            torch.cuda._sleep(20_000_000)  # the host gets ahead
        steps()
    torch.cuda.synchronize()
    assert m.status_read(ws[:4].view(torch.int32)) == 0
    codes = [t.view(torch.uint8) for t in (cache.k, cache.v)]
    ends = (starts0 + STEPS * add).tolist()
    assert max(ends) <= L
    bytes_ = [c[b, :, :n].clone() for c in codes for b, n in enumerate(ends)]
    scales = [s[b, :, :-(-n // BLOCK)].clone() for s in (cache.k_scale, cache.v_scale) for b, n in enumerate(ends)]
    return [o, ko, vo] + bytes_ + scales


@pytest.mark.parametrize("mode", ["queue", "graph"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("news", [[1, 1, 1, 1, 1], [5, 0, 2, 1, 8], [40, 3, 0, 17, 33], [80, 61, 1, 33, 50]])
def test_a_queue_of_calls_is_the_synchronised_run(moelib, cuda_dev, news, fmt, mode):
    want = _serve(moelib, fmt, news, "sync")
    assert all(torch.isfinite(t.float()).all() for t in want)
    for _ in range(3):
        for a, b in zip(want, _serve(moelib, fmt, news, mode)):
            assert torch.equal(a, b)
