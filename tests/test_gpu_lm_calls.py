"""How the language-model selections are called: derivatives, streams, host threads, messages."""
import ctypes as C
import threading

import pytest
import torch
import torch.autograd.forward_ad as fwd

pytestmark = pytest.mark.gpu


def rows(device, tokens=10, experts=16, seed=1):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randn((tokens, experts), generator=g, device=device), g


def test_forward_mode_is_refused(pk, cuda_device):
    z, g = rows(cuda_device)
    noise = torch.empty_like(z).exponential_(generator=g)
    one = torch.ones(10, device=cuda_device)
    r = pk.route(z, 2)
    dg, dl = torch.ones_like(r.gates), torch.ones((), device=cuda_device)
    with fwd.dual_level():
        dual = lambda t: fwd.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: pk.route(dual(z), 2), lambda: pk.sample_tokens(dual(z), noise),
                     lambda: pk.sample_tokens(z, noise, temperature=dual(one)),
                     lambda: pk.route_backward(dual(z), r, grad_gates=dg),
                     lambda: pk.route_backward(z, r, grad_gates=dual(dg)),
                     lambda: pk.route_backward(z, r, grad_gates=dg, grad_loss=dual(dl))):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        with pytest.raises(RuntimeError):
            pk.route(dual(z.clone().requires_grad_()), 2)
        # The choice does not vary with the noise or the bias, nor do the outputs.
        pk.sample_tokens(z, dual(noise))
        pk.route(z, 2, bias=dual(torch.ones(16, device=cuda_device)))
    assert torch.equal(pk.route(z, 2).gates, r.gates)


def test_function_transforms_are_refused(pk, cuda_device):
    z, g = rows(cuda_device)
    with pytest.raises(Exception):
        torch.func.jvp(lambda t: pk.route(t, 2).gates, (z,), (torch.ones_like(z),))
    with pytest.raises(Exception):
        torch.func.grad(lambda t: pk.route(t, 2).gates.square().sum())(z)
    with pytest.raises(Exception):
        torch.vmap(lambda t: pk.route(t, 2).gates)(z.expand(3, 10, 16))
    with pytest.raises(Exception):
        torch.vmap(lambda t: pk.sample_tokens(t, torch.ones_like(z))[0])(z.expand(3, 10, 16))


@pytest.mark.parametrize("of", ["gates", "loss"])
def test_a_second_derivative_raises(pk, cuda_device, of):
    z, _ = rows(cuda_device)
    z.requires_grad_()
    r = pk.route(z, 2, normalize=False)
    y = r.gates.sum() if of == "gates" else r.loss
    grad, = torch.autograd.grad(y, z, create_graph=True)
    with pytest.raises(NotImplementedError):
        (y * 0 + grad.square().sum()).backward()


def test_log_probabilities_come_without_a_graph(pk, cuda_device):
    z, g = rows(cuda_device)
    noise = torch.empty_like(z).exponential_(generator=g)
    want = pk.sample_tokens(z, noise)
    got = pk.sample_tokens(z.clone().requires_grad_(), noise)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not got[1].requires_grad


@pytest.mark.parametrize("call", ["sample_tokens", "route", "route_backward"])
def test_outputs_on_another_stream_leave_freed_blocks_alone(pk, cuda_device, call):
    # Inputs made on the side stream, which therefore has no reason to wait for the current one; there, work is
    # queued on tensors of the outputs' sizes that have been let go.  Outputs made from their memory would be
    # written before it is read.
    tokens, E, k = 4096, 64, 4
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        z, g = rows(cuda_device, tokens, E)
        noise = torch.empty_like(z).exponential_(generator=g)
        r = pk.route(z, k)
        dg = torch.ones_like(r.gates).cumsum(1)
        want = {"sample_tokens": lambda: pk.sample_tokens(z, noise), "route": lambda: pk.route(z, k)[:4],
                "route_backward": lambda: (pk.route_backward(z, r, grad_gates=dg),)}[call]()
    torch.cuda.synchronize()
    freed = [torch.full(t.shape, 7, dtype=t.dtype, device=cuda_device) for t in want]
    kept = [torch.zeros_like(t) for t in freed]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    for a, b in zip(kept, freed):
        a.copy_(b)
    blocks = {t.data_ptr() for t in freed}
    del freed, a, b
    got = {"sample_tokens": lambda: pk.sample_tokens(z, noise, stream=side), "route": lambda: pk.route(z, k, stream=side)[:4],
           "route_backward": lambda: (pk.route_backward(z, r, grad_gates=dg, stream=side),)}[call]()
    assert not blocks & {t.data_ptr() for t in got}
    side.synchronize()
    assert all(torch.equal(x.cpu(), y.cpu()) for x, y in zip(got, want))
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in kept)


def test_outputs_of_another_stream_outlive_their_use_here(pk, cuda_device):
    # Let go while the current stream still has work on them: the side stream must not get the memory yet.
    z, _ = rows(cuda_device, 4096, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = pk.route(z, 4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    kept, want = torch.zeros_like(r.gates), r.gates.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    kept.copy_(r.gates)
    block = r.gates.data_ptr()
    del r
    again = pk.route(z, 4, stream=side)
    assert block not in {t.data_ptr() for t in again[:4]}
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_streams_given_and_current_agree(pk, cuda_device):
    z, g = rows(cuda_device, 500, 64)
    noise = torch.empty_like(z).exponential_(generator=g)
    want, lp = pk.sample_tokens(z, noise, top_k=5)
    torch.cuda.synchronize()
    for stream in (torch.cuda.default_stream(), torch.cuda.current_stream(), torch.cuda.Stream(),
                   torch.cuda.ExternalStream(torch.cuda.Stream().cuda_stream)):
        before = torch.cuda.current_stream()
        got = pk.sample_tokens(z, noise, top_k=5, stream=stream)
        assert torch.cuda.current_stream() == before
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and torch.equal(got[1], lp)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = pk.sample_tokens(z, noise, top_k=5, stream=side)
        r = pk.route(z, 3, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    z.copy_(z.flip(0))
    graph.replay()
    want = pk.sample_tokens(z, noise, top_k=5)
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(r.experts, pk.route(z, 3).experts)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("wide,narrow", [(256, 130), (512, 260), (1024, 600)])
def test_host_threads_with_different_numbers_of_experts(pk, cuda_device, dtype, wide, narrow):
    # Both counts take the same kernels with different amounts of shared memory.  Through the C-ABI, whose calls
    # run side by side (ctypes gives up the interpreter's lock), each thread on a stream of its own.
    from streaming_selection_primitive_gb300 import _abi
    lib = pk.lib()

    def arrays(E):
        z, g = rows(cuda_device, 300, E, seed=E)
        z = z.to(dtype)
        out = [torch.empty((300, 4), device=cuda_device), torch.empty((300, 4), dtype=torch.int64, device=cuda_device),
               torch.empty(E, dtype=torch.int64, device=cuda_device), torch.empty((), device=cuda_device), torch.empty_like(z)]
        return z, out, torch.cuda.Stream()

    def work(E, z, out, stream, failed):
        how = _abi.Routing(_abi.SCORE_SIGMOID, 1)
        kind = _abi.F32 if dtype == torch.float32 else _abi.BF16
        gates, experts, counts, loss, grad = (t.data_ptr() for t in out)
        for i in range(3000):
            a = lib.profk_route(z.data_ptr(), kind, 300, E, E, 4, C.byref(how), gates, experts, counts, loss, stream.cuda_stream)
            b = lib.profk_route_backward(z.data_ptr(), kind, 300, E, E, 4, C.byref(how), experts, counts, gates, loss, grad, E,
                                         stream.cuda_stream)
            if a or b:
                failed.append((E, i, a, b))
                return

    sets = {E: arrays(E) for E in (wide, narrow)}
    torch.cuda.synchronize()
    failed = []
    threads = [threading.Thread(target=work, args=(E, *sets[E], failed)) for E in (wide, narrow)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for E, (z, out, _) in sets.items():
        r = pk.route(z, 4, score="sigmoid")
        assert torch.equal(out[0], r.gates) and torch.equal(out[1], r.experts) and torch.equal(out[2], r.counts)


def test_messages_say_what_is_wanted(pk, cuda_device):
    z, g = rows(cuda_device)  # 10 x 16
    noise = torch.empty_like(z).exponential_(generator=g)
    r = pk.route(z, 2)
    wide = torch.ones((10, 4), device=cuda_device)
    for call, error, words in (
            (lambda: pk.sample_tokens(z, noise, top_p=torch.ones(3, device=cuda_device)), ValueError, r"top_p must have shape \(10,\), not \(3,\)"),
            (lambda: pk.sample_tokens(z, noise, top_p=wide[:, 0]), ValueError, "top_p must be contiguous"),
            (lambda: pk.sample_tokens(z, noise[:, :5]), ValueError, r"noise must have shape \(10, 16\), not \(10, 5\)"),
            (lambda: pk.sample_tokens(z, noise.t().contiguous().t()), ValueError, "noise must have unit column stride"),
            (lambda: pk.sample_tokens(z, noise, mask=torch.ones((10, 2), dtype=torch.int32, device=cuda_device)), ValueError,
             r"mask must have shape \(10, 1\), not \(10, 2\)"),
            (lambda: pk.route(z, 2, bias=torch.ones(15, device=cuda_device)), ValueError, r"bias must have shape \(16,\), not \(15,\)"),
            (lambda: pk.route(z, 2, mask=torch.ones((10, 1), dtype=torch.bool, device=cuda_device)), ValueError,
             r"mask must have shape \(10,\), not \(10, 1\)"),
            (lambda: pk.route_backward(z, r, grad_gates=wide[:, :2]), ValueError, "grad_gates must be contiguous"),
            (lambda: pk.route_backward(z, r, grad_gates=wide), ValueError, r"grad_gates must have shape \(10, 2\), not \(10, 4\)"),
            (lambda: pk.route_backward(z[:5], r), ValueError, r"routing.experts must have shape \(5, 2\), not \(10, 2\)")):
        with pytest.raises(error, match=words):
            call()


def test_host_threads_through_python(pk, cuda_device):
    # Four threads, each with inputs and a stream of its own, sample, route and go backward.
    def work(i, out):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            z, g = rows(cuda_device, 200 + 50 * i, 40 + 30 * i, seed=i)
            noise = torch.empty_like(z).exponential_(generator=g)
            leaf = z.clone().requires_grad_()
            for _ in range(50):
                token, lp = pk.sample_tokens(z, noise, top_k=7, top_p=0.9)
                r = pk.route(leaf, 3)
                leaf.grad = None
                (r.gates.square().sum() + r.loss).backward()
            stream.synchronize()
            out[i] = [t.cpu() for t in (token, lp, r.gates.detach(), r.experts, r.counts, r.loss.detach(), leaf.grad)]

    alone, together = {}, {}
    for i in range(4):
        work(i, alone)
    threads = [threading.Thread(target=work, args=(i, together)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(a, b) for i in range(4) for a, b in zip(alone[i], together[i]))
